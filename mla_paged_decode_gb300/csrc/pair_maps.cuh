// The tensor maps of the pair kernel's loads of the cache.
#pragma once

#include <cuda.h>

namespace mla {

struct PairMaps {
  CUtensorMap k;   // one dim block of 128 bytes of a page's rows
  CUtensorMap k4;  // e4m3: the last 64 dims of a page's rows
  CUtensorMap v;   // one CTA's value dims of half a bf16 page, of an e4m3 page
  CUtensorMap va;  // the same of eight rows
  CUtensorMap vr;  // one dim block of one row
};

}  // namespace mla
