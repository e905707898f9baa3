// Latent attention and its cache: what the host code and the kernels share.
#ifndef KDACONV_LATENT_H_
#define KDACONV_LATENT_H_

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kdaconv.h"

namespace kdaconv {

constexpr int kLatentMax = 512;  // channels of a latent
constexpr int kRopeMax = 64;  // channels of a rotated part
constexpr int kScaleBlock = 32;  // channels that share a scale in the 8-bit cache

// n / d for 0 <= n < 2^31 by a multiplication and a shift (Granlund and Montgomery's round-up
// method).
struct Divider {
  uint32_t d, magic;
  int32_t shift;
  __host__ __device__ uint32_t operator()(uint32_t n) const {
    const uint32_t high = (uint32_t)(((uint64_t)n * magic) >> 32);
    return (high + n) >> shift;  // below 2^32: n < 2^31, high <= n
  }
};

inline Divider divider_of(uint32_t d) {
  int l = 0;
  while (((uint64_t)1 << l) < d) ++l;
  const unsigned __int128 num = (unsigned __int128)1 << (32 + l);
  return Divider{d, (uint32_t)((num + d - 1) / d - ((unsigned __int128)1 << 32)), l};
}

// A paged cache as the kernels see it; strides in bytes.
struct CacheView {
  char* latents;
  char* ropes;
  uint8_t* scales;
  int64_t lat_page, lat_slot, rope_page, rope_slot, scale_page, scale_slot;
  int32_t num_pages, latent, rope;
  Divider page_size;
};

// Sequences of a call, and the table of their pages.
struct PageTable {
  const int32_t* table;
  int64_t stride;
  int32_t width;  // pages per sequence
};

// Checks of a cache (sizes, strides and, with `pointers`, addresses) and its view.
int validate_cache(const kdaconv_latent_cache* c, bool pointers);
CacheView cache_view(const kdaconv_latent_cache* c);

}  // namespace kdaconv

#endif  // KDACONV_LATENT_H_
