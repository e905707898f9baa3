// Rotary positions, and the latent cache's write and read (include/kdaconv.h states all three).
//
// All are streams: what bounds them is HBM, or for the few tokens of a decode batch the launch.
#include "latent_device.h"

#include <algorithm>

namespace kdaconv {
namespace {

constexpr int kWave = 64;

// ------------------------------------------------------------------------------ rotary

struct RotaryParams {
  const char* x;
  char* out;
  const void* positions;
  const float* inv_freq;
  int64_t x_s0, x_s1, o_s0, o_s1;  // bytes
  int32_t tokens, heads, dim, rotary, offset;
  int32_t per_block;  // tokens of a workgroup
  float scale;
  bool positions_64, interleaved, rest_stays;
  Divider pairs, units, head_units, copy_units, head_copies;
};

constexpr int kRotaryThreads = 256, kAngles = 256;

// A workgroup's tokens share one table of angles, which its threads work out first: the sine
// and cosine in FP64 reduction cost some 150 instructions, once per token and pair rather than
// once per head. Then a thread turns `units` of kV channels (kV = 8: 16 bytes a load). 16384 tokens
// of 12 heads, 64 channels turned in place: 9.6 us, 5.3 TB/s of the 64; 37 tokens 4 us, a launch.
template <int kF, int kV>
__global__ __launch_bounds__(kRotaryThreads) void rotary_kernel(RotaryParams P) {
  __shared__ f32x2 table[kAngles];
  constexpr int kE = elem_bytes<kF>();
  const int first = blockIdx.x * P.per_block;
  const int count = P.tokens - first < P.per_block ? P.tokens - first : P.per_block;
  const int pairs = P.rotary / 2;
  for (int i = threadIdx.x; i < count * pairs; i += kRotaryThreads) {
    const int t = P.pairs(i), j = i - t * pairs;
    const f32x2 cs = turn(load_index(P.positions, first + t, P.positions_64), P.inv_freq[j]);
    table[i] = f32x2{P.scale * cs.x, P.scale * cs.y};
  }
  __syncthreads();
  const int units = P.units.d;
  for (int i = threadIdx.x; i < count * P.heads * units; i += kRotaryThreads) {
    const int t = P.head_units(i), rest = i - t * (P.heads * units);
    const int h = P.units(rest), u = rest - h * units;
    const char* const x = P.x + (first + t) * P.x_s0 + h * P.x_s1 + P.offset * kE;
    char* const o = P.out + (first + t) * P.o_s0 + h * P.o_s1 + P.offset * kE;
    const f32x2* const cs = table + t * pairs;
    if constexpr (kV == 8) {
      if (P.interleaved) {
        float v[8];
        load_eight<kF>(x + u * 8 * kE, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const f32x2 r = turned(v[2 * j], v[2 * j + 1], cs[4 * u + j]);
          v[2 * j] = r.x;
          v[2 * j + 1] = r.y;
        }
        store_eight<kF>(o + u * 8 * kE, v);
      } else {
        float a[8], b[8];
        load_eight<kF>(x + u * 8 * kE, a);
        load_eight<kF>(x + (pairs + u * 8) * kE, b);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const f32x2 r = turned(a[j], b[j], cs[8 * u + j]);
          a[j] = r.x;
          b[j] = r.y;
        }
        store_eight<kF>(o + u * 8 * kE, a);
        store_eight<kF>(o + (pairs + u * 8) * kE, b);
      }
    } else {
      const int at = P.interleaved ? 2 * u : u, to = P.interleaved ? 2 * u + 1 : pairs + u;
      const f32x2 r = turned(load_elem<kF>(x + at * kE), load_elem<kF>(x + to * kE), cs[u]);
      store_elem<kF>(o + at * kE, r.x);
      store_elem<kF>(o + to * kE, r.y);
    }
  }
  if (P.rest_stays) return;
  const int copies = P.copy_units.d;  // of the other channels; a head without any is never here
  for (int i = threadIdx.x; i < count * P.heads * copies; i += kRotaryThreads) {
    const int t = P.head_copies(i), rest = i - t * (P.heads * copies);
    const int h = P.copy_units(rest);
    int c = (rest - h * copies) * kV;
    if (c >= P.offset) c += P.rotary;
    const char* const x = P.x + (first + t) * P.x_s0 + h * P.x_s1 + c * kE;
    char* const o = P.out + (first + t) * P.o_s0 + h * P.o_s1 + c * kE;
    if constexpr (kV == 8) {
      if constexpr (kF == kRuleF32) {
        const f32x4 a = ((const f32x4a4*)x)[0], b = ((const f32x4a4*)x)[1];
        ((f32x4a4*)o)[0] = a;
        ((f32x4a4*)o)[1] = b;
      } else {
        *(u32x4_any*)o = *(const u32x4_any*)x;
      }
    } else if constexpr (kF == kRuleF32) {
      *(uint32_t*)o = *(const uint32_t*)x;
    } else {
      *(uint16_t*)o = *(const uint16_t*)x;
    }
  }
}

template <int kF>
void launch_rotary(const RotaryParams& P, bool wide, int64_t blocks, hipStream_t st) {
  if (wide)
    hipLaunchKernelGGL((rotary_kernel<kF, 8>), dim3((unsigned)blocks), dim3(kRotaryThreads), 0, st, P);
  else
    hipLaunchKernelGGL((rotary_kernel<kF, 1>), dim3((unsigned)blocks), dim3(kRotaryThreads), 0, st, P);
}

// ------------------------------------------------------------------------------- write

struct WriteParams {
  CacheView C;
  const char* latent;
  const char* rope;
  const void* slots;
  const float* weight;
  const void* positions;
  const float* inv_freq;
  int64_t latent_stride, rope_stride;  // bytes
  double eps, inv_dim;
  int32_t tokens;
  float rope_scale;
  bool norm, slots_64, positions_64, interleaved;
};

constexpr int kWriteWaves = 4;

// One wave per token, 8 channels of the latent per lane. A block of 32 channels is four lanes.
// Latency bounds it: a wave's row, then an FP64 sum over six lane exchanges, a division and a root,
// then the stores, with nothing else of the wave's to do meanwhile. 16384 tokens of 512 + 64 bf16
// channels take 11.5 to 12 us (3.2 TB/s) and 13 into 8 bits (2.2 TB/s), 37 tokens 4 us, a launch.
template <int kF, bool kE4m3>
__global__ __launch_bounds__(kWave * kWriteWaves) void latent_write_kernel(WriteParams P) {
  const int lane = threadIdx.x % kWave;
  const int t = uniform(blockIdx.x * kWriteWaves + threadIdx.x / kWave);
  if (t >= P.tokens) return;
  const int c = lane * 8;
  const bool mine = c < P.C.latent;
  float x[8] = {};
  if (mine) load_eight<kF>(P.latent + t * P.latent_stride + c * 2, x);
  // The rotated part: one pair per lane.
  const int pairs = P.C.rope / 2;
  const bool turns = lane < pairs;
  const bool adjacent = P.interleaved || P.inv_freq == nullptr;
  const int u = adjacent ? 2 * lane : lane, v = adjacent ? 2 * lane + 1 : pairs + lane;
  f32x2 r = {0.0f, 0.0f};
  if (turns) {
    const char* const row = P.rope + t * P.rope_stride;
    r = f32x2{load_elem<kF>(row + u * 2), load_elem<kF>(row + v * 2)};
    if (P.inv_freq != nullptr) {
      const f32x2 cs = turn(load_index(P.positions, t, P.positions_64), P.inv_freq[lane]);
      r = turned(r.x, r.y, f32x2{P.rope_scale * cs.x, P.rope_scale * cs.y});
    }
  }
  float w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = 1.0f;
  if (mine && P.weight != nullptr) load_eight<kRuleF32>((const char*)(P.weight + c), w);
  const int64_t slot = load_index(P.slots, t, P.slots_64);
  if (slot < 0 || slot >= (int64_t)P.C.num_pages * P.C.page_size.d) return;  // the whole wave
  const uint32_t page = P.C.page_size((uint32_t)slot), at = (uint32_t)slot - page * P.C.page_size.d;

  if (P.norm) {
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = __builtin_fma((double)x[i], (double)x[i], sum);
    sum = lane_sum<kWave>(sum);
    const double f = 1.0 / __builtin_sqrt(sum * P.inv_dim + P.eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)((double)x[i] * f * (double)w[i]);
  }
  char* const to = P.C.latents + page * P.C.lat_page + at * P.C.lat_slot;
  if constexpr (kE4m3) {
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = __builtin_fabsf(x[i]);
      most = is_finite(a) ? __builtin_fmaxf(most, a) : most;
    }
    most = __builtin_fmaxf(most, __shfl_xor(most, 1));
    most = __builtin_fmaxf(most, __shfl_xor(most, 2));
    const int byte = scale_byte(most);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] = is_finite(x[i]) ? __builtin_amdgcn_ldexpf(x[i], 127 - byte) : __builtin_nanf("");
    u32x2 codes;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      int pack = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * i], x[4 * i + 1], 0, false);
      codes[i] = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * i + 2], x[4 * i + 3], pack, true);
    }
    if (mine) {
      *(u32x2*)(to + c) = codes;
      if (lane % 4 == 0) P.C.scales[page * P.C.scale_page + at * P.C.scale_slot + lane / 4] = (uint8_t)byte;
    }
  } else {
    if (mine) *(u32x4*)(to + c * 2) = pack_eight<kF>(x);
  }
  if (turns) {
    char* const row = P.C.ropes + page * P.C.rope_page + at * P.C.rope_slot;
    store_elem<kF>(row + u * 2, r.x);
    store_elem<kF>(row + v * 2, r.y);
  }
}

// -------------------------------------------------------------------------------- read

struct ReadParams {
  CacheView C;
  PageTable T;
  const int32_t* starts;
  char* out;
  int32_t tokens, seqs, search_top;
  int32_t row_chunks;  // of 8 channels
  int32_t per;  // rows of a wave, up to 64
  Divider chunks;
};

constexpr int kReadWaves = 4, kReadAhead = 2;

// A wave reads some neighbouring rows of the output: its lanes first find each row's sequence and
// slot, then copy 8 channels at a time, kReadAhead loads before the first is waited for. Memory
// bounds it: 131072 rows of 512 8-bit and 64 16-bit channels take 46 to 49 us among calls of their
// kind, 237 MB at 5 TB/s, and 62 us after other work has filled the caches (one load at a time 63 us
// where this took 49, six 67: registers then leave fewer waves); 16-bit rows, 302 MB, take 54 us.
template <int kF, bool kE4m3>
__global__ __launch_bounds__(kWave * kReadWaves) void latent_read_kernel(ReadParams P) {
  const int lane = threadIdx.x % kWave;
  const int first = uniform((blockIdx.x * kReadWaves + threadIdx.x / kWave) * P.per);
  if (first >= P.tokens) return;
  // The last sequence that starts at or before the first row; 64-way search, a ballot a level.
  int s = 0;
  for (int stride = P.search_top; stride > 0; stride >>= 6) {
    const int at = s + lane * stride;
    const uint64_t mask = __ballot(at < P.seqs && P.starts[at] <= first);
    const int n = __builtin_popcountll(mask);
    if (n == 0) break;  // before the first sequence
    s += (n - 1) * stride;
  }
  // Row `lane` of the wave's: its slot, -1 for zeros, -2 for a row that no sequence owns.
  int64_t slot = -2;
  const int row = first + lane;
  if (lane < P.per && row < P.tokens) {
    int mine = s;
    while (mine < P.seqs && P.starts[mine + 1] <= row) ++mine;
    if (mine < P.seqs && P.starts[mine] <= row) {
      const uint32_t i = row - std::max(0, P.starts[mine]), p = P.C.page_size(i);
      slot = -1;
      if ((int64_t)p < P.T.width) {
        const int page = P.T.table[mine * P.T.stride + p];
        if (page >= 0 && page < P.C.num_pages) slot = (int64_t)page * P.C.page_size.d + (i - p * P.C.page_size.d);
      }
    }
  }
  const int latent_chunks = P.C.latent / 8, total = P.per * P.row_chunks;
  for (int base = lane; base < total; base += kWave * kReadAhead) {
    u32x4 v[kReadAhead];
    uint32_t scales[kReadAhead];
    char* to[kReadAhead];
    bool codes[kReadAhead];
#pragma unroll
    for (int u = 0; u < kReadAhead; ++u) {
      const int i = base + u * kWave;
      const int t = P.chunks(i), c = i - t * P.row_chunks;
      const int at = i < total ? __shfl((int)slot, t) : -2;
      v[u] = u32x4{0, 0, 0, 0};
      scales[u] = 127;
      to[u] = at == -2 ? nullptr : P.out + ((int64_t)(first + t) * P.row_chunks + c) * 16;
      codes[u] = kE4m3 && c < latent_chunks;
      if (at >= 0) {
        const uint32_t page = P.C.page_size((uint32_t)at), place = (uint32_t)at - page * P.C.page_size.d;
        if (c >= latent_chunks) {
          v[u] = *(const u32x4*)(P.C.ropes + page * P.C.rope_page + place * P.C.rope_slot + (c - latent_chunks) * 16);
        } else if constexpr (!kE4m3) {
          v[u] = *(const u32x4*)(P.C.latents + page * P.C.lat_page + place * P.C.lat_slot + c * 16);
        } else {
          const u32x2 q = *(const u32x2*)(P.C.latents + page * P.C.lat_page + place * P.C.lat_slot + c * 8);
          v[u][0] = q[0], v[u][1] = q[1];
          scales[u] = P.C.scales[page * P.C.scale_page + place * P.C.scale_slot + c / 4];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kReadAhead; ++u) {
      if (kE4m3 && codes[u]) {
        const float f = scale_value(scales[u]);
        const uint32_t lo = v[u][0], hi = v[u][1];
        v[u] = u32x4{scaled_pair<kF, false>(lo, f), scaled_pair<kF, true>(lo, f),
                     scaled_pair<kF, false>(hi, f), scaled_pair<kF, true>(hi, f)};
      }
      if (to[u] != nullptr) *(u32x4*)to[u] = v[u];
    }
  }
}

bool aligned_to(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

}  // namespace

int validate_cache(const kdaconv_latent_cache* c, bool pointers) {
  if (c == nullptr) return KDACONV_EINVAL;
  if (c->num_pages < 0 || c->page_size <= 0 || c->latent_dim <= 0 || c->rope_dim < 0) return KDACONV_EINVAL;
  if (c->dtype != KDACONV_BF16 && c->dtype != KDACONV_F16 && c->dtype != KDACONV_F32) return KDACONV_EINVAL;
  if (c->dtype == KDACONV_F32) return KDACONV_EUNSUPPORTED;
  const int64_t block = c->e4m3 ? kScaleBlock : 8, bytes = c->e4m3 ? 1 : 2;
  if (c->latent_dim % block != 0 || c->latent_dim > kLatentMax) return KDACONV_EUNSUPPORTED;
  if (c->rope_dim % 8 != 0 || c->rope_dim > kRopeMax) return KDACONV_EUNSUPPORTED;
  if (c->page_size > INT32_MAX || c->num_pages > INT32_MAX || c->num_pages * c->page_size > INT32_MAX)
    return KDACONV_EUNSUPPORTED;
  // Strides of axes of one entry mean nothing.
  const bool pages = c->num_pages > 1, slots = c->page_size > 1;
  if ((pages && c->latents_stride0 < 0) || (slots && c->latents_stride1 < 0) ||
      (pages && c->latents_stride0 * bytes % 16) || (slots && c->latents_stride1 * bytes % 16))
    return KDACONV_EUNSUPPORTED;
  if (c->rope_dim > 0 &&
      ((pages && c->ropes_stride0 < 0) || (slots && c->ropes_stride1 < 0) ||
       (pages && c->ropes_stride0 * 2 % 16) || (slots && c->ropes_stride1 * 2 % 16)))
    return KDACONV_EUNSUPPORTED;
  if (c->e4m3 && ((pages && c->scales_stride0 < 0) || (slots && c->scales_stride1 < 0)))
    return KDACONV_EUNSUPPORTED;
  if (pointers && c->num_pages > 0) {
    if (!c->latents || (c->rope_dim > 0 && !c->ropes) || (c->e4m3 && !c->scales)) return KDACONV_EINVAL;
    if (!aligned_to(c->latents, 16) || (c->rope_dim > 0 && !aligned_to(c->ropes, 16)))
      return KDACONV_EUNSUPPORTED;
  }
  return KDACONV_OK;
}

CacheView cache_view(const kdaconv_latent_cache* c) {
  CacheView v;
  v.latents = static_cast<char*>(c->latents);
  v.ropes = static_cast<char*>(c->ropes);
  v.scales = c->scales;
  const int64_t bytes = c->e4m3 ? 1 : 2, pages = c->num_pages > 1, slots = c->page_size > 1;
  v.lat_page = c->latents_stride0 * bytes * pages;
  v.lat_slot = c->latents_stride1 * bytes * slots;
  v.rope_page = c->ropes_stride0 * 2 * pages;
  v.rope_slot = c->ropes_stride1 * 2 * slots;
  v.scale_page = c->scales_stride0 * pages;
  v.scale_slot = c->scales_stride1 * slots;
  v.num_pages = (int32_t)c->num_pages;
  v.latent = (int32_t)c->latent_dim;
  v.rope = (int32_t)c->rope_dim;
  v.page_size = divider_of((uint32_t)c->page_size);
  return v;
}

}  // namespace kdaconv

using namespace kdaconv;

extern "C" int kdaconv_rotary_embedding(const void* x, int dtype, int64_t num_tokens, int64_t num_heads,
                                        int64_t head_dim, int64_t x_stride0, int64_t x_stride1,
                                        const void* positions, int positions_64, const float* inv_freq,
                                        int64_t rotary, int64_t offset, int interleaved, double scale,
                                        void* out, int64_t out_stride0, int64_t out_stride1,
                                        kdaconv_stream_t stream) {
  if (num_tokens < 0 || num_heads < 0 || head_dim <= 0) return KDACONV_EINVAL;
  if (dtype != KDACONV_BF16 && dtype != KDACONV_F16 && dtype != KDACONV_F32) return KDACONV_EINVAL;
  if (rotary <= 0 || rotary % 2 != 0 || offset < 0 || rotary > head_dim || offset > head_dim - rotary)
    return KDACONV_EINVAL;
  if (rotary > 2 * kAngles) return KDACONV_EUNSUPPORTED;
  // Strides of axes of one entry mean nothing.
  const int64_t tokens = num_tokens > 1, heads = num_heads > 1;
  x_stride0 *= tokens, out_stride0 *= tokens, x_stride1 *= heads, out_stride1 *= heads;
  if (x_stride0 < 0 || x_stride1 < 0 || out_stride0 < 0 || out_stride1 < 0) return KDACONV_EUNSUPPORTED;
  // Each element of out is written: heads of a token, and tokens, may not overlap.
  if ((heads && out_stride1 < head_dim) || (tokens && out_stride0 < head_dim)) return KDACONV_EINVAL;
  if (num_tokens > INT32_MAX / 2 || num_heads > 65535 || head_dim > 65536) return KDACONV_EUNSUPPORTED;
  if (num_tokens == 0 || num_heads == 0) return KDACONV_OK;
  if (!x || !out || !positions || !inv_freq) return KDACONV_EINVAL;
  const int64_t e = dtype == KDACONV_F32 ? 4 : 2;
  if (!aligned_to(x, e) || !aligned_to(out, e) || !aligned_to(inv_freq, 4) ||
      !aligned_to(positions, positions_64 ? 8 : 4))
    return KDACONV_EUNSUPPORTED;
  RotaryParams P;
  P.x = static_cast<const char*>(x);
  P.out = static_cast<char*>(out);
  P.positions = positions;
  P.inv_freq = inv_freq;
  P.x_s0 = x_stride0 * e;
  P.x_s1 = x_stride1 * e;
  P.o_s0 = out_stride0 * e;
  P.o_s1 = out_stride1 * e;
  P.tokens = (int32_t)num_tokens;
  P.heads = (int32_t)num_heads;
  P.dim = (int32_t)head_dim;
  P.rotary = (int32_t)rotary;
  P.offset = (int32_t)offset;
  P.scale = (float)scale;
  P.positions_64 = positions_64 != 0;
  P.interleaved = interleaved != 0;
  const int64_t others = head_dim - rotary;
  P.rest_stays = others == 0 || (x == out && P.x_s0 == P.o_s0 && P.x_s1 == P.o_s1);
  // Units of 8 channels where the parts are made of them.
  const bool wide = rotary % (interleaved ? 8 : 16) == 0 && (P.rest_stays || (offset % 8 == 0 && others % 8 == 0));
  const int64_t units = wide ? (interleaved ? rotary / 8 : rotary / 16) : rotary / 2;
  const int64_t copies = std::max<int64_t>(1, wide ? others / 8 : others);
  // Tokens of a workgroup: as many as its table holds, but no more than leave 1024 workgroups,
  // four per CU.
  const int64_t most = std::max<int64_t>(1, kAngles / (rotary / 2));
  P.per_block = (int32_t)std::max<int64_t>(1, std::min(most, num_tokens / 1024));
  // A workgroup's units are counted in 31 bits, a stride past their end too.
  if (P.per_block * num_heads * std::max(units, copies) > INT32_MAX - kRotaryThreads) return KDACONV_EUNSUPPORTED;
  P.pairs = divider_of((uint32_t)(rotary / 2));
  P.units = divider_of((uint32_t)units);
  P.head_units = divider_of((uint32_t)(units * num_heads));
  P.copy_units = divider_of((uint32_t)copies);
  P.head_copies = divider_of((uint32_t)(copies * num_heads));
  const int64_t blocks = (num_tokens + P.per_block - 1) / P.per_block;
  if (blocks >= (int64_t)1 << 24) return KDACONV_EUNSUPPORTED;  // 2^32 threads
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (dtype == KDACONV_F32)
    launch_rotary<kRuleF32>(P, wide, blocks, st);
  else if (dtype == KDACONV_F16)
    launch_rotary<kRuleF16>(P, wide, blocks, st);
  else
    launch_rotary<kRuleBF16>(P, wide, blocks, st);
  return hipGetLastError() == hipSuccess ? KDACONV_OK : KDACONV_ELAUNCH;
}

extern "C" int kdaconv_latent_cache_write(const kdaconv_latent_cache* cache, const void* latent,
                                          int64_t latent_stride, const void* rope, int64_t rope_stride,
                                          int64_t num_tokens, const void* slots, int slots_64,
                                          const float* weight, double eps, const void* positions,
                                          int positions_64, const float* inv_freq, int interleaved,
                                          double rope_scale, kdaconv_stream_t stream) {
  const int rc = validate_cache(cache, num_tokens > 0);
  if (rc != KDACONV_OK) return rc;
  if (num_tokens < 0 || eps != eps) return KDACONV_EINVAL;
  if (num_tokens > INT32_MAX / 2) return KDACONV_EUNSUPPORTED;
  latent_stride *= num_tokens > 1, rope_stride *= num_tokens > 1;
  if (latent_stride < 0 || rope_stride < 0) return KDACONV_EUNSUPPORTED;
  // The cache's places may not overlap: each is written.
  const bool pages = cache->num_pages > 1, places = cache->page_size > 1;
  if ((places && cache->latents_stride1 < cache->latent_dim) || (pages && cache->latents_stride0 < cache->latent_dim) ||
      (places && cache->ropes_stride1 < cache->rope_dim) || (pages && cache->ropes_stride0 < cache->rope_dim))
    return KDACONV_EINVAL;
  const int64_t blocks_of_scales = cache->latent_dim / kScaleBlock;
  if (cache->e4m3 && ((places && cache->scales_stride1 < blocks_of_scales) || (pages && cache->scales_stride0 < blocks_of_scales)))
    return KDACONV_EINVAL;
  if (num_tokens == 0 || cache->num_pages == 0) return KDACONV_OK;
  if (!latent || (cache->rope_dim > 0 && !rope) || !slots || (inv_freq && !positions)) return KDACONV_EINVAL;
  if (!aligned_to(latent, 2) || !aligned_to(rope, 2) || !aligned_to(weight, 4) || !aligned_to(inv_freq, 4) ||
      !aligned_to(slots, slots_64 ? 8 : 4) || !aligned_to(positions, positions_64 ? 8 : 4))
    return KDACONV_EUNSUPPORTED;
  WriteParams P;
  P.C = cache_view(cache);
  P.latent = static_cast<const char*>(latent);
  P.rope = static_cast<const char*>(rope);
  P.slots = slots;
  P.weight = weight;
  P.positions = positions;
  P.inv_freq = inv_freq;
  P.latent_stride = latent_stride * 2;
  P.rope_stride = rope_stride * 2;
  P.eps = eps;
  P.inv_dim = 1.0 / (double)cache->latent_dim;
  P.tokens = (int32_t)num_tokens;
  P.rope_scale = (float)rope_scale;
  P.norm = eps >= 0.0;
  P.slots_64 = slots_64 != 0;
  P.positions_64 = positions_64 != 0;
  P.interleaved = interleaved != 0;
  const int64_t blocks = (num_tokens + kWriteWaves - 1) / kWriteWaves;
  if (blocks >= (int64_t)1 << 24) return KDACONV_EUNSUPPORTED;  // 2^32 threads
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  const dim3 grid((unsigned)blocks), block(kWave * kWriteWaves);
  if (cache->dtype == KDACONV_BF16 && cache->e4m3)
    hipLaunchKernelGGL((latent_write_kernel<kRuleBF16, true>), grid, block, 0, st, P);
  else if (cache->dtype == KDACONV_BF16)
    hipLaunchKernelGGL((latent_write_kernel<kRuleBF16, false>), grid, block, 0, st, P);
  else if (cache->e4m3)
    hipLaunchKernelGGL((latent_write_kernel<kRuleF16, true>), grid, block, 0, st, P);
  else
    hipLaunchKernelGGL((latent_write_kernel<kRuleF16, false>), grid, block, 0, st, P);
  return hipGetLastError() == hipSuccess ? KDACONV_OK : KDACONV_ELAUNCH;
}

extern "C" int kdaconv_latent_cache_read(const kdaconv_latent_cache* cache, const int32_t* block_table,
                                         int64_t table_stride, int64_t pages_per_seq,
                                         const int32_t* kv_start_loc, int64_t num_seqs,
                                         int64_t num_tokens, void* out, kdaconv_stream_t stream) {
  const int rc = validate_cache(cache, num_tokens > 0 && num_seqs > 0);
  if (rc != KDACONV_OK) return rc;
  if (num_tokens < 0 || num_seqs < 0 || pages_per_seq < 0) return KDACONV_EINVAL;
  table_stride *= num_seqs > 1;
  if (table_stride < 0 || num_tokens > INT32_MAX / 2 || num_seqs > INT32_MAX / 2 || pages_per_seq > INT32_MAX)
    return KDACONV_EUNSUPPORTED;
  if (num_tokens == 0 || num_seqs == 0) return KDACONV_OK;
  if (!kv_start_loc || !out || (pages_per_seq > 0 && !block_table)) return KDACONV_EINVAL;
  if (!aligned_to(kv_start_loc, 4) || !aligned_to(block_table, 4) || !aligned_to(out, 16))
    return KDACONV_EUNSUPPORTED;
  ReadParams P;
  P.C = cache_view(cache);
  P.T = PageTable{block_table, table_stride, (int32_t)pages_per_seq};
  P.starts = kv_start_loc;
  P.out = static_cast<char*>(out);
  P.tokens = (int32_t)num_tokens;
  P.seqs = (int32_t)num_seqs;
  int64_t reach = kWave;
  while (reach < num_seqs) reach *= kWave;
  P.search_top = (int32_t)(reach / kWave);
  P.row_chunks = (int32_t)((cache->latent_dim + cache->rope_dim) / 8);
  P.chunks = divider_of((uint32_t)P.row_chunks);
  // 16 rows a wave, or 4 where that leaves CUs without 4 waves: 4004 rows, written and read, 10.4 us
  // in a graph and 21.9 with 16; 131072 rows 67 and 60.
  P.per = num_tokens >= 256 * 4 * 16 ? 16 : 4;
  const int64_t per = P.per * kReadWaves, blocks = (num_tokens + per - 1) / per;
  if (blocks >= (int64_t)1 << 24) return KDACONV_EUNSUPPORTED;  // 2^32 threads
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  const dim3 grid((unsigned)blocks), block(kWave * kReadWaves);
  if (cache->dtype == KDACONV_BF16 && cache->e4m3)
    hipLaunchKernelGGL((latent_read_kernel<kRuleBF16, true>), grid, block, 0, st, P);
  else if (cache->dtype == KDACONV_BF16)
    hipLaunchKernelGGL((latent_read_kernel<kRuleBF16, false>), grid, block, 0, st, P);
  else if (cache->e4m3)
    hipLaunchKernelGGL((latent_read_kernel<kRuleF16, true>), grid, block, 0, st, P);
  else
    hipLaunchKernelGGL((latent_read_kernel<kRuleF16, false>), grid, block, 0, st, P);
  return hipGetLastError() == hipSuccess ? KDACONV_OK : KDACONV_ELAUNCH;
}
