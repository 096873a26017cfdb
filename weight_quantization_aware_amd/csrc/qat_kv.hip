// A served decoder block's attention (gfx950, wave64): rotary positions, the
// paged 8-bit cache of keys and values, and the attention that reads it.
#include <math.h>

#include <type_traits>

#include "../../include/qat_kv.h"
#include "qat_check.h"
#include "qat_device.h"
#include "qat_internal.h"

namespace qat {
namespace {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

template <int DT>
struct Half8;                       // 8 elements of the activations' type
template <>
struct Half8<QAT_BF16> {
  typedef bf16x8 v;
};
template <>
struct Half8<QAT_F16> {
  typedef f16x8 v;
};

template <int DT>
__device__ __forceinline__ float to_float(uint32_t bits16) {
  if constexpr (DT == QAT_BF16) return __builtin_bit_cast(float, bits16 << 16);
  else return (float)__builtin_bit_cast(_Float16, (uint16_t)bits16);
}

template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (DT == QAT_BF16) return pack_bf16x2(a, b);
  else return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b});
}

template <int DT>
__device__ __forceinline__ void unpack8(uint4 v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[2 * j] = to_float<DT>(w[j] & 0xFFFFu);
    x[2 * j + 1] = to_float<DT>(w[j] >> 16);
  }
}

template <int DT>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack2<DT>(x[0], x[1]), pack2<DT>(x[2], x[3]), pack2<DT>(x[4], x[5]), pack2<DT>(x[6], x[7]));
}

// ---------------------------------------------------------------------------
// Rotary positions. A workgroup owns one token and a share of its heads: the
// token's rot / 2 angles are formed once, in 64 bits (a far position times a
// frequency loses every fractional bit in 32), reduced to [-pi, pi] and put
// into LDS as cosine and sine; then each thread turns 16 elements (two 16-byte
// loads) of a head. Bound by HBM for prompts (4096 tokens of 64 + 8 heads in 29
// us, 5.2 TB/s), by the launch for single tokens.
// ---------------------------------------------------------------------------
struct RopeArgs {
  const uint16_t* q;
  const uint16_t* k;
  uint16_t* qo;
  uint16_t* ko;
  const int32_t* pos;
  const float* inv_freq;
  int64_t ldq, ldk, ldqo, ldko;
  int hq, hk, d, rot, half;
  int pieces;                      // 16-element pieces of a head
  float mscale, sign;
};

template <int DT>
__global__ __launch_bounds__(256) void k_rope(const RopeArgs a) {
  __shared__ float cs[64], sn[64];
  const int64_t t = blockIdx.x;
  const int half_rot = a.rot / 2;
  if (threadIdx.x < half_rot) {
    const double ang = (double)a.pos[t] * (double)a.inv_freq[threadIdx.x];
    const double n = rint(ang * 0.15915494309189533577);           // 1 / (2 pi)
    // 2 pi as a double and the rest of it
    const float r = (float)fma(-n, 2.4492935982947064e-16, fma(-n, 6.283185307179586232, ang));
    cs[threadIdx.x] = cosf(r) * a.mscale;
    sn[threadIdx.x] = sinf(r) * (a.mscale * a.sign);
  }
  __syncthreads();
  const int total = (a.hq + a.hk) * a.pieces;
  const int turned = a.rot / 16;                                   // pieces that turn; the rest is copied
  for (int i = blockIdx.y * 256 + threadIdx.x; i < total; i += gridDim.y * 256) {
    const int h = i / a.pieces, p = i - h * a.pieces;
    const bool is_q = h < a.hq;
    const uint16_t* src = is_q ? a.q + t * a.ldq + h * a.d : a.k + t * a.ldk + (h - a.hq) * a.d;
    uint16_t* dst = is_q ? a.qo + t * a.ldqo + h * a.d : a.ko + t * a.ldko + (h - a.hq) * a.d;
    const bool split = a.half && p < turned;                       // pairs half_rot apart
    const int e0 = split ? 8 * p : 16 * p, e1 = split ? 8 * p + half_rot : 16 * p + 8;
    uint4 u = *(const uint4*)(src + e0), v = *(const uint4*)(src + e1);
    if (p < turned) {
      float x[8], y[8], xo[8], yo[8];
      unpack8<DT>(u, x);
      unpack8<DT>(v, y);
      const float* c = cs + 8 * p;
      const float* s = sn + 8 * p;
      if (a.half) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          xo[j] = x[j] * c[j] - y[j] * s[j];
          yo[j] = y[j] * c[j] + x[j] * s[j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          xo[2 * j] = x[2 * j] * c[j] - x[2 * j + 1] * s[j];
          xo[2 * j + 1] = x[2 * j + 1] * c[j] + x[2 * j] * s[j];
          yo[2 * j] = y[2 * j] * c[4 + j] - y[2 * j + 1] * s[4 + j];
          yo[2 * j + 1] = y[2 * j + 1] * c[4 + j] + y[2 * j] * s[4 + j];
        }
      }
      u = pack8<DT>(xo);
      v = pack8<DT>(yo);
    }
    *(uint4*)(dst + e0) = u;
    *(uint4*)(dst + e1) = v;
  }
}

// ---------------------------------------------------------------------------
// Append. A workgroup owns one (page, head) block of the keys or the values of
// one sequence: it reads the block's new tokens once into registers, finds
// their largest finite magnitude, sets the block's scale, rounds the earlier
// tokens' codes again where the scale grew, and writes the new codes. Values
// go through LDS, which turns [token][d] into the cache's [d][token]. Bound by
// HBM for prompts (2 x 2048 tokens of 32 heads in 22 us, 4.2 TB/s), by four
// dependent loads for single tokens (7 us).
// ---------------------------------------------------------------------------
struct AppendArgs {
  const uint16_t* x[2];            // keys, values
  int64_t ld[2];
  uint8_t* cache[2];
  float* scale[2];
  const int32_t* cu;
  const int32_t* lens;
  const int32_t* table;
  int64_t cols, tokens, n_pages, max_new;
  int heads, d, page;
};

// Four codes times f, rounded again.
__device__ __forceinline__ uint32_t requant4(uint32_t c, float f) {
  const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, true);
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(a[0] * f, a[1] * f, 0, false);
  r = __builtin_amdgcn_cvt_pk_fp8_f32(b[0] * f, b[1] * f, r, true);
  return (uint32_t)r;
}

template <int DT, int NT, int PASSES>
__global__ __launch_bounds__(NT) void k_kv_append(const AppendArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];   // values: [d][page + 4]
  __shared__ uint32_t wave_max[NT / 64];
  const int b = blockIdx.y, h = blockIdx.z >> 1, is_v = blockIdx.z & 1;
  const int64_t c0 = min(max((int64_t)a.cu[b], (int64_t)0), a.tokens);
  const int64_t c1 = min(max((int64_t)a.cu[b + 1], c0), a.tokens);
  const int64_t start = (int64_t)a.lens[b] - (c1 - c0);            // position of token c0
  const int64_t lo_pos = max(start, (int64_t)0);
  const int64_t hi_pos = min(start + min(c1 - c0, a.max_new), a.cols * a.page);
  if (lo_pos >= hi_pos) return;
  const int64_t blk = lo_pos / a.page + blockIdx.x, base = blk * a.page;
  if (base >= hi_pos) return;
  const int64_t pid = a.table[b * a.cols + blk];
  if (pid < 0 || pid >= a.n_pages) return;
  const int lo = (int)(max(lo_pos, base) - base), hi = (int)(min(hi_pos, base + a.page) - base);   // new slots
  const int per = a.d / 8;                                         // 16-byte pieces of a token
  const int npiece = (hi - lo) * per;
  const int64_t row0 = c0 + (base + lo - start);
  const uint16_t* x = a.x[is_v] + h * a.d;
  const int64_t ld = a.ld[is_v];

  uint4 v[PASSES];
  uint32_t amax = 0;
  constexpr uint32_t kOdd = DT == QAT_BF16 ? 0x7F80u : 0x7C00u;    // infinities and NaN from here on
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int p = i * NT + threadIdx.x;
    v[i] = make_uint4(0, 0, 0, 0);
    if (p < npiece) v[i] = *(const uint4*)(x + (row0 + p / per) * ld + (p % per) * 8);
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t m0 = w[j] & 0x7FFFu, m1 = (w[j] >> 16) & 0x7FFFu;
      amax = max(amax, max(m0 < kOdd ? m0 : 0u, m1 < kOdd ? m1 : 0u));
    }
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) amax = max(amax, (uint32_t)__shfl_xor((int)amax, o));
  if constexpr (NT > 64) {
    if ((threadIdx.x & 63) == 0) wave_max[threadIdx.x >> 6] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) amax = max(amax, wave_max[w]);
  }
  // the smallest e with 448 2^e >= amax: floor(log2 amax) - 8, one more above 1.75 2^floor
  const uint32_t mb = __builtin_bit_cast(uint32_t, to_float<DT>(amax));
  int e = max((int)(mb >> 23) - 135 + ((mb & 0x7FFFFFu) > 0x600000u ? 1 : 0), -126);
  float* scale = a.scale[is_v] + pid * a.heads + h;
  float again = 1.0f;                                              // what earlier codes are multiplied by
  if (lo > 0) {
    const int e_old = min((int)((__builtin_bit_cast(uint32_t, *scale) >> 23) & 255u) - 127, 126);
    if (e_old >= e) {
      e = e_old;
    } else {
      const int d = e_old - e;
      again = d > -127 ? __builtin_bit_cast(float, (uint32_t)(127 + d) << 23) : 0.0f;
    }
  }
  e = max(e, -126);
  const float inv = __builtin_bit_cast(float, (uint32_t)(127 - e) << 23);
  uint8_t* cache = a.cache[is_v] + (pid * a.heads + h) * (int64_t)a.page * a.d;

  if constexpr (NT > 64) __syncthreads();                          // everyone has read *scale
  if (threadIdx.x == 0) *scale = __builtin_bit_cast(float, (uint32_t)(127 + e) << 23);

  uint32_t code[PASSES][2];
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    float f[8];
    unpack8<DT>(v[i], f);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = __builtin_fabsf(f[j]) < INFINITY ? f[j] * inv : NAN;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      int c = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * j], f[4 * j + 1], 0, false);
      c = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * j + 2], f[4 * j + 3], c, true);
      code[i][j] = (uint32_t)c;
    }
  }
  if (!is_v) {
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int p = i * NT + threadIdx.x;
      if (p < npiece) *(uint2*)(cache + lo * a.d + p * 8) = make_uint2(code[i][0], code[i][1]);
    }
    if (again != 1.0f) {
      for (int p = threadIdx.x; p < lo * a.d / 16; p += NT) {
        uint4* c = (uint4*)cache + p;
        const uint4 u = *c;
        *c = make_uint4(requant4(u.x, again), requant4(u.y, again), requant4(u.z, again), requant4(u.w, again));
      }
    }
    return;
  }
  const int pitch = a.page + 4;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int p = i * NT + threadIdx.x;
    if (p < npiece) {
      uint8_t* dst = smem + (p % per) * 8 * pitch + lo + p / per;
#pragma unroll
      for (int j = 0; j < 8; ++j) dst[j * pitch] = (uint8_t)(code[i][j >> 2] >> (8 * (j & 3)));
    }
  }
  __syncthreads();
  // 16 slots of one d at a time; the block belongs to this workgroup alone, so
  // a piece that also holds earlier or later slots is read, changed and written
  const int pieces = a.page / 16;
  for (int p = threadIdx.x; p < a.d * pieces; p += NT) {
    const int dd = p / pieces, s0 = (p - dd * pieces) * 16;
    const bool any_new = s0 < hi && s0 + 16 > lo, any_old = again != 1.0f && s0 < lo;
    if (!any_new && !any_old) continue;
    uint32_t* c = (uint32_t*)(cache + dd * a.page + s0);
    const uint32_t* n = (const uint32_t*)(smem + dd * pitch + s0);
    if (s0 >= lo && s0 + 16 <= hi) {
      *(uint4*)c = make_uint4(n[0], n[1], n[2], n[3]);
    } else if (again == 1.0f) {
      for (int s = max(lo, s0); s < min(hi, s0 + 16); ++s) ((uint8_t*)c)[s - s0] = smem[dd * pitch + s];
    } else {
      const uint4 u = *(const uint4*)c;
      const uint32_t old[4] = {u.x, u.y, u.z, u.w};
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t re = requant4(old[j], again), nw = any_new ? n[j] : 0u;
        uint32_t r = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int s = s0 + 4 * j + k;
          r |= ((s < lo ? re : s < hi ? nw : old[j]) >> (8 * k) & 255u) << (8 * k);
        }
        w[j] = r;
      }
      *(uint4*)c = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// ---------------------------------------------------------------------------
// Attention over the cache, few rows. A row is one (token, head) pair; the
// rows of one sequence that share a key head are packed 16 to an MFMA tile, so
// a key or value byte is read once for all of them. Bound by HBM: 2 head_dim
// bytes for each cached position and key head.
//
// Each wave takes blocks of 64 positions on its own, from global memory
// straight into registers, without LDS or barriers in the loop:
//   S^T = K Q^T: lane (r16 = 4 a + r, g) of tile jt holds key 16 a + 4 jt + r,
//     bytes head_dim / 4 g .. (any order of d does, Q takes the same), codes
//     made exact bf16 or fp16 of Q's type; the result lane then has, for its
//     row r16, keys 16 g + 4 jt + r: 16 consecutive positions of one page, so
//     one key scale and one value scale a lane;
//   O^T += V^T P^T: the lane's 16 probabilities are the B operand as they sit;
//     the A operand, d = 16 jd + r16 and the same 16 positions, is 16
//     consecutive bytes of the cache's [d][token] value block.
// The softmax runs with a lazily moved row maximum in base 2; a lane asks with
// its own positions' maximum whether it has to move, and the lanes of a row
// join theirs only then. A probability is multiplied by its page's value scale
// over a reference (the largest so far) and rounded to fp16: 11 bits, against
// bf16's 8, and e4m3 is exact in fp16. The product of the two is at most 2^12;
// what falls below fp16's 2^-24 is 2^-24 of the largest weight of the row.
// ---------------------------------------------------------------------------
struct AttnArgs {
  const uint16_t* q;
  int64_t ldq;
  const int32_t* cu;
  const int32_t* lens;
  const int32_t* table;
  int64_t cols, tokens, n_pages;
  int batch, hk, group, log_page;
  const uint8_t* k;
  const uint8_t* v;
  const float* ks;
  const float* vs;
  float scale_log2;                // softmax_scale log2(e)
  int causal;
  int64_t max_new, max_len;
  uint16_t* out;
  int64_t ldo;
  int target;                      // workgroups of a key head; 0: one for each sequence
  int max_rows;                    // max_new * group
  int row_blocks;                  // of a sequence and key head (prompts)
  float* part_o;                   // [part][key head][max_rows][head_dim]
  float* part_ml;                  // [part][key head][max_rows][2]
};

constexpr int kTile = 64;          // positions of a block
constexpr int kMinTiles = 8;       // blocks of a run at least: two for each of a workgroup's four waves
constexpr float kLazy = 8.0f;      // how far (log2) a block's maximum may pass the subtracted one
constexpr float kLazyV = 4.0f;     // the same of value scales over their reference
constexpr float kMostSum = 32768.0f; // of a lane's 16 weights, each a fp16 number then
constexpr float kLowC = -40.0f;    // log2 of a value scale over the reference is held at this or more

struct Seq {
  int64_t c0;                      // first new token
  int n;                           // new tokens
  int64_t start;                   // their first position
  int len;                         // cached positions
};

__device__ __forceinline__ Seq seq_of(const AttnArgs& a, int b) {
  Seq s;
  s.c0 = min(max((int64_t)a.cu[b], (int64_t)0), a.tokens);
  const int64_t c1 = min(max((int64_t)a.cu[b + 1], s.c0), a.tokens);
  const int64_t len = a.lens[b];
  s.start = len - (c1 - s.c0);
  s.n = (int)min(c1 - s.c0, a.max_new);
  s.len = (int)max(min(min(len, a.max_len), a.cols << a.log_page), (int64_t)0);
  return s;
}

// Blocks of a sequence; one at least, so that the rows of a sequence without
// positions are someone's too.
__device__ __forceinline__ int tiles_of(const AttnArgs& a, int b) {
  const int64_t len = max(min(min((int64_t)a.lens[b], a.max_len), a.cols << a.log_page), (int64_t)0);
  return max((int)((len + kTile - 1) / kTile), 1);
}

__device__ __forceinline__ int wave_sum(int v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o);
  return v;
}

// The blocks of all sequences, one sequence after the other, are dealt to the
// workgroups of a key head in equal runs, whatever the lengths; a run may end one
// sequence and begin others. Every wave finds its way for itself.
// Blocks before sequence b (of all with b = batch).
__device__ __forceinline__ int64_t tiles_before(const AttnArgs& a, int b) {
  const int lane = threadIdx.x & 63;
  int64_t n = 0;
  for (int b0 = 0; b0 < b; b0 += 64) n += wave_sum(b0 + lane < b ? tiles_of(a, b0 + lane) : 0);
  return n;
}

__device__ __forceinline__ int64_t run_length(const AttnArgs& a, int64_t total) {
  const int64_t n = (total + a.target - 1) / a.target;
  return n > kMinTiles ? n : kMinTiles;
}

// The sequence that block `at` (below the total) is in, and the blocks before it.
__device__ __forceinline__ int seq_at(const AttnArgs& a, int64_t at, int64_t& before) {
  const int lane = threadIdx.x & 63;
  before = 0;
  for (int b0 = 0; b0 < a.batch; b0 += 64) {
    const int cnt = b0 + lane < a.batch ? tiles_of(a, b0 + lane) : 0;
    int inc = cnt;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int up = __shfl_up(inc, o);
      if (lane >= o) inc += up;
    }
    const uint64_t past = __ballot(before + inc > at);
    if (past) {
      const int l = __builtin_ctzll(past);
      before += __shfl(inc - cnt, l);
      return b0 + l;
    }
    before += __shfl(inc, 63);
  }
  return a.batch - 1;
}

// Largest value over the four lanes that share lane & 15.
__device__ __forceinline__ float max_over_g(float x) {
  x = fmaxf(x, __shfl_xor(x, 16));
  return fmaxf(x, __shfl_xor(x, 32));
}

// 8 codes (two dwords) as bf16 or fp16.
template <int DT>
__device__ __forceinline__ typename Half8<DT>::v codes8(uint32_t lo, uint32_t hi) {
  if constexpr (DT == QAT_BF16) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
  } else {
    const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
    const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
    const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
    const f16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
    return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
  }
}

__device__ __forceinline__ f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma16(f16x8 a, f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// Takes the values that are not numbers out of 8 fp16 values (zero in their
// place) and returns 1 for each of them, 0 for the others. On the bits, two at
// a time: compared one by one, the 128 truth values of a block would not fit
// the scalar registers.
__device__ __forceinline__ f16x8 take_nan(f16x8& v) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  u32x4 u = __builtin_bit_cast(u32x4, v), n;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    // above 0x7C00 without the sign: the sum carries into bit 15
    const uint32_t top = ((u[j] & 0x7FFF7FFFu) + 0x03FF03FFu) & 0x80008000u;
    const uint32_t mask = (top >> 15) * 0xFFFFu;
    u[j] &= ~mask;
    n[j] = mask & 0x3C003C00u;
  }
  v = __builtin_bit_cast(f16x8, u);
  return __builtin_bit_cast(f16x8, n);
}

// 1 for the first `n` of 8 fp16 values, 0 for the others.
__device__ __forceinline__ f16x8 ones8(int n) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  u32x4 u;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int k = min(max(n - 2 * j, 0), 2);
    u[j] = 0x3C003C00u & (uint32_t)((1ull << (16 * k)) - 1);
  }
  return __builtin_bit_cast(f16x8, u);
}

// Whether one of 16 codes is not a number.
__device__ __forceinline__ bool has_nan(uint4 u) {
  const uint32_t k7 = 0x7F7F7F7Fu, k1 = 0x01010101u;
  return ((((u.x & k7) + k1) | ((u.y & k7) + k1) | ((u.z & k7) + k1) | ((u.w & k7) + k1)) & 0x80808080u) != 0;
}

// What a key page's scale and the softmax's make of a score, for a lane whose
// positions hold `have` keys: positive, so that the maximum can be taken before
// it, and never zero, so that a masked score stays -inf. A scale that is not a
// number stays one; that of a page left out does not matter.
__device__ __forceinline__ float score_factor(float key_scale, float scale_log2, int have) {
  const float f = have > 0 ? key_scale * scale_log2 : 1.0f;
  return f < 0x1p-126f ? 0x1p-126f : f;
}

// log2 of a value page's scale over the reference, at kLowC or more (also where
// both are zero).
__device__ __forceinline__ float scale_over(float lv, float vref, int have) {
  const float d = lv - vref;
  return have <= 0 ? 0.0f : lv != lv ? lv : d > kLowC ? d : kLowC;
}

// The first `n` (0 .. 16) bytes of 16, the others zero.
__device__ __forceinline__ uint4 first_bytes(uint4 u, int n) {
  uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int k = min(max(n - 4 * j, 0), 4);
    w[j] &= k == 4 ? 0xFFFFFFFFu : (1u << (8 * k)) - 1u;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int DT, int D>
__global__ __launch_bounds__(256, 2) void k_kv_decode(const AttnArgs a) {
  typedef typename Half8<DT>::v half8;
  constexpr int RT = 1;                                  // row tiles of a wave; two spill at head_dim 128
  constexpr int KP = D / 64, JD = D / 16, KS = D / 32;
  constexpr int kPitch = D + 4;
  __shared__ __attribute__((aligned(16))) float so[4][16][kPitch];
  __shared__ float sm[4][16], sl[4][16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int h = blockIdx.y;
  // this workgroup's run of blocks: [at, end), in sequence b behind `before`
  int b = blockIdx.x;
  int64_t at_block = 0, end_block = 0, before = 0;
  if (a.target) {
    const int64_t total = tiles_before(a, a.batch), run = run_length(a, total);
    at_block = (int64_t)blockIdx.x * run;
    if (at_block >= total) return;
    end_block = min(at_block + run, total);
    b = seq_at(a, at_block, before);
  }
  bool first_seq = true;
  do {
    b = __builtin_amdgcn_readfirstlane(b);
    const Seq s = seq_of(a, b);
    const int row_base = blockIdx.z * 16 * RT;
    const int rows = s.n * a.group;
    const int all = max((s.len + kTile - 1) / kTile, 1);   // as tiles_of
    const int t0 = a.target ? __builtin_amdgcn_readfirstlane((int)(at_block - before)) : 0;
    const int t_end = a.target ? __builtin_amdgcn_readfirstlane((int)min(end_block - before, (int64_t)all)) : all;
    const bool whole = t0 == 0 && t_end == all;
    at_block = before + t_end;
    before += all;
    if (row_base < rows) {
      if (!first_seq) __syncthreads();                       // the last sequence's parts have been read from LDS
      first_seq = false;

      // this lane's rows, their limits (positions below are seen) and queries
      half8 qf[RT][KS];
      int lim[RT], lo_lim = 0x7FFFFFFF, hi_lim = 0;
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const int row = row_base + 16 * i + r16;
        const int rc = min(row, rows - 1);
        const int tok = rc / a.group, hh = rc - tok * a.group;
        const int64_t seen = a.causal ? s.start + tok + 1 : (int64_t)s.len;
        lim[i] = (int)max(min(seen, (int64_t)s.len), (int64_t)0);
        lo_lim = min(lo_lim, lim[i]);
        hi_lim = max(hi_lim, lim[i]);
        const uint16_t* qp = a.q + (s.c0 + tok) * a.ldq + (int64_t)(h * a.group + hh) * D + D / 4 * g;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) qf[i][ks] = *(const half8*)(qp + 8 * ks);
      }
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) {
        lo_lim = min(lo_lim, __shfl_xor(lo_lim, o));
        hi_lim = max(hi_lim, __shfl_xor(hi_lim, o));
      }
      lo_lim = __builtin_amdgcn_readfirstlane(lo_lim);
      hi_lim = __builtin_amdgcn_readfirstlane(hi_lim);
      const int t1 = min(t_end, (hi_lim + kTile - 1) / kTile);
      const bool one_limit = lo_lim == hi_lim;

      const int32_t* table = a.table + b * a.cols;
      const int page = 1 << a.log_page;
      const int last16 = max(s.len - 1, 0) >> 4;             // the last 16 positions that hold any
      const int64_t head_bytes = (int64_t)page * D;

      // A block's keys and values are in registers once: the next block's keys are
      // loaded as soon as the scores have been formed, its values as soon as the
      // output has been, so each load has the other half of a block's work and
      // the next scores to arrive in.
      // Page ids of the two 16-position groups a lane loads from: r16 / 4 for
      // keys, g for values and scales.
      auto page_of = [&](int t, int sub) { return table[(min(4 * t + sub, last16) << 4) >> a.log_page]; };
      uint4 xk[4][KP], xv[JD];
      float xks = 0.f, xvs = 0.f;      // scales of the lane's 16 positions
      int have = 0;                    // how many of them the cache holds (0: none, or a page left out)
      int id_a = 0, id_g = 0;          // pages of the block to load next
      auto load_k = [&](int t) {
        const int sub = min(4 * t + (r16 >> 2), last16);
        const int64_t blk = (int64_t)((uint32_t)id_a < (uint64_t)a.n_pages ? id_a : 0) * a.hk + h;
        const uint8_t* kp = a.k + blk * head_bytes + (int64_t)(((sub << 4) & (page - 1)) + (r16 & 3)) * D + D / 4 * g;
#pragma unroll
        for (int jt = 0; jt < 4; ++jt)
#pragma unroll
          for (int p = 0; p < KP; ++p) xk[jt][p] = *(const uint4*)(kp + 4 * jt * D + 16 * p);
      };
      auto load_v = [&](int t) {
        const bool bad = (uint32_t)id_g >= (uint64_t)a.n_pages;
        const int sub = min(4 * t + g, last16);
        const int64_t blk = (int64_t)(bad ? 0 : id_g) * a.hk + h;
        const uint8_t* vp = a.v + blk * head_bytes + ((sub << 4) & (page - 1)) + r16 * page;
#pragma unroll
        for (int jd = 0; jd < JD; ++jd) xv[jd] = *(const uint4*)(vp + 16 * jd * page);
        xks = a.ks[blk];
        xvs = a.vs[blk];
        have = bad ? 0 : min(max(s.len - 64 * t - 16 * g, 0), 16);
      };

      f32x4 o[RT][JD];
      float m[RT], l[RT];                                    // l: this lane's share of the row's sum
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int jd = 0; jd < JD; ++jd) o[i][jd] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
      float vref = -INFINITY;                                // log2 of the value scales' reference, wave-uniform

      auto compute = [&](int t, bool more) {
        // some position of the block is masked for some row, absent, or in a page left out
        const bool edge = 64 * t + 64 > lo_lim || __any(have < 16);
        f32x4 sc[RT][4];
#pragma unroll
        for (int jt = 0; jt < 4; ++jt) {
#pragma unroll
          for (int i = 0; i < RT; ++i) sc[i][jt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            const uint4 u = xk[jt][ks >> 1];
            const half8 kf = (ks & 1) ? codes8<DT>(u.z, u.w) : codes8<DT>(u.x, u.y);
#pragma unroll
            for (int i = 0; i < RT; ++i) sc[i][jt] = mfma16(kf, qf[i][ks], sc[i][jt]);
          }
        }
        if (more) load_k(t + 4);
        const float f = score_factor(xks, a.scale_log2, have);
        const int key0 = 64 * t + 16 * g;
        float mx[RT];
        bool grow = false;
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          if (edge) {
            const int seen = min(lim[i] - key0, have);       // of the lane's 16 positions
#pragma unroll
            for (int jt = 0; jt < 4; ++jt)
#pragma unroll
              for (int r = 0; r < 4; ++r)
                if (4 * jt + r >= seen) sc[i][jt][r] = -INFINITY;
          }
          float y = sc[i][0][0];
#pragma unroll
          for (int jt = 0; jt < 4; ++jt)
#pragma unroll
            for (int r = 0; r < 4; ++r) y = fmaxf(y, sc[i][jt][r]);
          mx[i] = y * f;                                     // of the lane's positions: enough to ask
          grow = grow || mx[i] > m[i] + kLazy;
        }
        const float lv = have > 0 ? __builtin_amdgcn_logf(xvs) : -INFINITY;
        if (__any(grow || lv > vref + kLazyV)) {
          const float lvm = max_over_g(lv), vn = lvm > vref + kLazyV ? lvm : vref;
          const float fv = vref == vn ? 1.0f : __builtin_amdgcn_exp2f(vref - vn);
          vref = vn;
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            const float mn = fmaxf(m[i], max_over_g(mx[i]));
            const float al = m[i] == mn ? 1.0f : __builtin_amdgcn_exp2f(m[i] - mn);
            l[i] *= al;
            m[i] = mn;
#pragma unroll
            for (int jd = 0; jd < JD; ++jd)
#pragma unroll
              for (int r = 0; r < 4; ++r) o[i][jd][r] *= al * fv;
          }
        }
        // w = 2^(s f + log2 c - m), c the lane's value scale over the reference; the
        // softmax's sum takes 1 / c once for the lane's 16 positions
        const float lc = scale_over(lv, vref, have);
        const float rc = __builtin_amdgcn_exp2f(-lc);
        f16x8 pf[RT][2];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          // a row that has seen nothing yet has m = -inf: its scores are all -inf
          const float ms = lc - (m[i] == -INFINITY ? 0.0f : m[i]);
          float sum = 0.f;
#pragma unroll
          for (int jt = 0; jt < 4; ++jt)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[i][jt][r], f, ms));
              sum += w;
              pf[i][jt >> 1][4 * (jt & 1) + r] = (_Float16)w;
            }
          l[i] += sum * rc;
        }
        if (!edge) {
#pragma unroll
          for (int jd = 0; jd < JD; ++jd) {
            const f16x8 v0 = codes8<QAT_F16>(xv[jd].x, xv[jd].y), v1 = codes8<QAT_F16>(xv[jd].z, xv[jd].w);
#pragma unroll
            for (int i = 0; i < RT; ++i) o[i][jd] = mfma16(v1, pf[i][1], mfma16(v0, pf[i][0], o[i][jd]));
          }
        } else {
          // Absent positions' values are zeroed whatever they hold. Where the rows'
          // limits differ, a value that is not a number may be seen by one row and
          // masked for another: it is taken out of the product, and counted apart
          // against the positions that each row sees.
          const int keep = one_limit ? min(lo_lim - key0, have) : have;
#pragma unroll
          for (int jd = 0; jd < JD; ++jd) {
            const uint4 u = first_bytes(xv[jd], keep);
            f16x8 v0 = codes8<QAT_F16>(u.x, u.y), v1 = codes8<QAT_F16>(u.z, u.w);
            if (!one_limit) {
              const f16x8 n0 = take_nan(v0), n1 = take_nan(v1);
#pragma unroll
              for (int i = 0; i < RT; ++i) {
                const int seen = min(lim[i] - key0, have);
                const f32x4 cnt = mfma16(n1, ones8(seen - 8), mfma16(n0, ones8(seen), f32x4{0.f, 0.f, 0.f, 0.f}));
#pragma unroll
                for (int r = 0; r < 4; ++r) o[i][jd][r] = cnt[r] > 0.f ? NAN : o[i][jd][r];
              }
            }
#pragma unroll
            for (int i = 0; i < RT; ++i) o[i][jd] = mfma16(v1, pf[i][1], mfma16(v0, pf[i][0], o[i][jd]));
          }
        }
        if (more) {
          load_v(t + 4);
          if (t + 8 < t1) {
            id_a = page_of(t + 8, r16 >> 2);
            id_g = page_of(t + 8, g);
          }
        }
      };

      int t = t0 + wave;
      if (t < t1) {
        id_a = page_of(t, r16 >> 2);
        id_g = page_of(t, g);
        load_k(t);
        load_v(t);
        if (t + 4 < t1) {
          id_a = page_of(t + 4, r16 >> 2);
          id_g = page_of(t + 4, g);
        }
        for (; t < t1; t += 4) compute(t, t + 4 < t1);
      }

      // the four waves meet in LDS, 16 rows at a time
      const float vscale = vref == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(vref);
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        if (i) __syncthreads();
#pragma unroll
        for (int jd = 0; jd < JD; ++jd) {
          const f32x4 v = o[i][jd];
          *(f32x4*)&so[wave][r16][16 * jd + 4 * g] = f32x4{v[0] * vscale, v[1] * vscale, v[2] * vscale, v[3] * vscale};
        }
        float row_sum = l[i];
        row_sum += __shfl_xor(row_sum, 16);
        row_sum += __shfl_xor(row_sum, 32);
        if (g == 0) {
          sm[wave][r16] = m[i];
          sl[wave][r16] = row_sum;
        }
        __syncthreads();
        const int rr = threadIdx.x >> 4, d0 = (threadIdx.x & 15) * (D / 16);
        const int row = row_base + 16 * i + rr;
        if (row >= rows) continue;
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < 4; ++w) mm = fmaxf(mm, sm[w][rr]);
        float ll = 0.f, acc[D / 16];
#pragma unroll
        for (int j = 0; j < D / 16; ++j) acc[j] = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          if (sl[w][rr] == 0.f) continue;                    // saw nothing
          const float f = __builtin_amdgcn_exp2f(sm[w][rr] - mm);
          ll += sl[w][rr] * f;
#pragma unroll
          for (int j = 0; j < D / 16; ++j) acc[j] += so[w][rr][d0 + j] * f;
        }
        if (whole) {
          const float inv = ll == 0.f ? 0.0f : 1.0f / ll;
          const int tok = row / a.group, hh = row - tok * a.group;
          uint16_t* op = a.out + (s.c0 + tok) * a.ldo + (int64_t)(h * a.group + hh) * D + d0;
#pragma unroll
          for (int j = 0; j < D / 16; j += 2) *(uint32_t*)(op + j) = pack2<DT>(acc[j] * inv, acc[j + 1] * inv);
        } else {
          // part (workgroup + sequence): along the runs one of the two grows from part to part
          const int64_t at = ((int64_t)((int)blockIdx.x + b) * a.hk + h) * a.max_rows + row;
#pragma unroll
          for (int j = 0; j < D / 16; j += 4)
            *(f32x4*)(a.part_o + at * D + d0 + j) = f32x4{acc[j], acc[j + 1], acc[j + 2], acc[j + 3]};
          if (d0 == 0) *(f32x2*)(a.part_ml + at * 2) = f32x2{mm, ll};
        }
      }
    }
    ++b;
  } while (a.target && at_block < end_block);
}

// ---------------------------------------------------------------------------
// Attention over the cache, many rows (prompts). A workgroup of four waves owns
// 128 rows of one (sequence, key head) and visits the blocks of 64 positions
// that they see. A block's codes are made 16-bit once for all rows
// and put into LDS (two buffers; the next block's codes are in flight in
// registers during this one's products); the products and the layout of a
// lane's scores are those of k_kv_decode. Bound by the matrix cores and, close
// behind, by the softmax's vector work, which is kept to a maximum, an FMA, an
// exponential and a sum for each score: the row maximum and both page scales
// are one FMA's constants. (A page's value scale over the reference is held at
// 2^-40 or more: below that the fp16 weights are zero either way.)
//
// Two prompts of 2048 tokens, 32 heads of 128: 92 us, 670 TFLOP/s of the seen
// pairs. Two waves a SIMD (256 registers) leave latency in the open.
//
// LDS: keys [64][D], 16-byte chunk c of key k at c ^ (k & 3 | k >> 2 & 12) (its
// lowest three bits for the 8 chunks of D = 64), values [D][64], chunk c of row
// d at c ^ (d & 7): fragment reads use every bank equally.
// ---------------------------------------------------------------------------
template <int D>
__device__ __forceinline__ int key_chunk(int key, int c) {
  const int sw = (key & 3) | (key >> 2 & 12);
  return D == 128 ? c ^ sw : c ^ (sw & 7);
}

template <int DT, int D>
__global__ __launch_bounds__(256, 2) void k_kv_prompt(const AttnArgs a) {
  typedef typename Half8<DT>::v half8;
  constexpr int NW = 4, RT = 2, JD = D / 16, KS = D / 32, kRows = 16 * RT * NW, NT = 64 * NW;
  constexpr int kBuf = 64 * D * 2;                       // bytes of one operand's block
  constexpr int NP = 4 * D / NT;                         // 16-byte pieces of a thread, each operand
  __shared__ __attribute__((aligned(1024))) uint8_t smem[2][2][kBuf];   // [buffer][keys, values]
  // values that are not numbers (rare): whether wave w put one, and where: bit j
  // of row d for position j, written by the rows' wave when it did
  __shared__ __attribute__((aligned(16))) int nan_of[2][NW];
  __shared__ __attribute__((aligned(8))) uint16_t nan_at[2][D][4];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  // (row block, sequence and head), the longest (last) row blocks of all heads
  // first: in the order of heads, the last heads' long blocks began last, and a
  // third of the time the chip was not full. Workgroups go to the 8 XCDs in
  // turn, so a head stays on one where the heads are a multiple of 8.
  const int probs = a.batch * a.hk, w = blockIdx.x;
  const int rb = a.row_blocks - 1 - w / probs, prob = w % probs;
  const int b = prob / a.hk, h = prob - b * a.hk;
  const Seq s = seq_of(a, b);
  const int rows = s.n * a.group, row_base = rb * kRows;
  if (row_base >= rows) return;

  // this lane's rows (16 i + r16 of its wave's), their limits and queries
  half8 qf[RT][KS];
  int lim[RT], lo_lim = 0x7FFFFFFF, hi_lim = 0;
  const int wave_base = row_base + wave * 16 * RT;
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int rc = min(wave_base + 16 * i + r16, rows - 1);
    const int tok = rc / a.group, hh = rc - tok * a.group;
    const int64_t seen = a.causal ? s.start + tok + 1 : (int64_t)s.len;
    lim[i] = (int)max(min(seen, (int64_t)s.len), (int64_t)0);
    lo_lim = min(lo_lim, lim[i]);
    hi_lim = max(hi_lim, lim[i]);
    const uint16_t* qp = a.q + (s.c0 + tok) * a.ldq + (int64_t)(h * a.group + hh) * D + 8 * g;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) qf[i][ks] = *(const half8*)(qp + 32 * ks);
  }
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) {
    lo_lim = min(lo_lim, __shfl_xor(lo_lim, o));
    hi_lim = max(hi_lim, __shfl_xor(hi_lim, o));
  }
  lo_lim = __builtin_amdgcn_readfirstlane(lo_lim);
  hi_lim = __builtin_amdgcn_readfirstlane(hi_lim);       // of the wave
  // limits grow with the row: the workgroup's last row sees most
  const int last_tok = (min(row_base + kRows, rows) - 1) / a.group;
  const int64_t most = a.causal ? min(s.start + last_tok + 1, (int64_t)s.len) : (int64_t)s.len;
  const int tiles = (int)((max(most, (int64_t)0) + kTile - 1) / kTile);

  const int32_t* table = a.table + b * a.cols;
  const int page = 1 << a.log_page, last16 = max(s.len - 1, 0) >> 4;
  const uint32_t head_bytes = (uint32_t)(page * D);
  auto page_of = [&](int t, int sub) { return table[(min(4 * t + sub, last16) << 4) >> a.log_page]; };
  auto block_of = [&](int id, bool& bad) {
    bad = (uint32_t)id >= (uint64_t)a.n_pages;
    return (uint32_t)(bad ? 0 : id) * (uint32_t)a.hk + (uint32_t)h;      // below 2^31 (checked)
  };

  // Staging: piece p = i NT + tid is 16 codes: keys' d 16 (p % (D / 16)) .. of
  // key p / (D / 16), and values' positions 16 (p % 4) .. of row d = p / 4.
  const int sub_v = tid & 3;                             // NT is a multiple of 4
  const uint8_t* kbase = a.k + (tid % JD) * 16;
  const uint8_t* vbase = a.v + (tid >> 2) * page;
  uint4 rk[NP], rv[NP];
  float nks = 0.f, nvs = 0.f;                            // the lane's 16 positions' scales, of the block in flight
  int nhave = 0, nkeep = 0;
  // Page ids are fetched a block ahead of the loads that need them.
  int id_k[NP], id_v, id_s;
  auto load_ids = [&](int t) {
#pragma unroll
    for (int i = 0; i < NP; ++i) id_k[i] = page_of(t, (i * NT + tid) / JD >> 4);
    id_v = page_of(t, sub_v);
    id_s = page_of(t, g);
  };
  auto load = [&](int t) {
    bool bad;
    const int rest = last16 - 4 * t;                     // 16-position groups behind the block's first
    const int in_page = 64 * t & (page - 1);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int key = (i * NT + tid) / JD;
      const uint32_t blk = block_of(id_k[i], bad);
      const int slot = ((in_page + (min(key >> 4, rest) << 4)) & (page - 1)) + (key & 15);
      rk[i] = *(const uint4*)(kbase + (uint64_t)blk * head_bytes + (uint32_t)(slot * D));
    }
    const uint32_t blk = block_of(id_v, bad);
    const uint8_t* vp = vbase + (uint64_t)blk * head_bytes + (uint32_t)((in_page + (min(sub_v, rest) << 4)) & (page - 1));
    nkeep = bad ? 0 : s.len - 64 * t - 16 * sub_v;
#pragma unroll
    for (int i = 0; i < NP; ++i) rv[i] = *(const uint4*)(vp + i * (NT / 4) * page);
    const uint32_t bg = block_of(id_s, bad);
    nks = a.ks[bg];
    nvs = a.vs[bg];
    nhave = bad ? 0 : min(max(s.len - 64 * t - 16 * g, 0), 16);
  };
  auto put = [&](int buf) {
    bool nan = false;
    if (__any(nkeep < 16)) {                             // absent positions' values are zero whatever they hold
#pragma unroll
      for (int i = 0; i < NP; ++i) rv[i] = first_bytes(rv[i], nkeep);
    }
#pragma unroll
    for (int i = 0; i < NP; ++i) nan = nan || has_nan(rv[i]);
    const bool any = __any(nan);
    if (lane == 0) nan_of[buf][wave] = any;
    if (any) {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        uint32_t u[4] = {rv[i].x, rv[i].y, rv[i].z, rv[i].w}, at = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t top = ((u[j] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
          u[j] &= ~((top >> 7) * 255u);
          at |= (((top >> 7) * 0x01020408u) >> 24 & 15u) << (4 * j);
        }
        rv[i] = make_uint4(u[0], u[1], u[2], u[3]);
        nan_at[buf][i * (NT / 4) + (tid >> 2)][tid & 3] = (uint16_t)at;
      }
    }
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int p = i * NT + tid, key = p / JD, c = (p % JD) * 2;
      uint8_t* kr = smem[buf][0] + key * (2 * D);
      *(half8*)(kr + key_chunk<D>(key, c) * 16) = codes8<DT>(rk[i].x, rk[i].y);
      *(half8*)(kr + key_chunk<D>(key, c + 1) * 16) = codes8<DT>(rk[i].z, rk[i].w);
      const int d = p >> 2, cv = (p & 3) * 2;
      uint8_t* vr = smem[buf][1] + d * 128;
      *(f16x8*)(vr + ((cv ^ (d & 7)) << 4)) = codes8<QAT_F16>(rv[i].x, rv[i].y);
      *(f16x8*)(vr + (((cv + 1) ^ (d & 7)) << 4)) = codes8<QAT_F16>(rv[i].z, rv[i].w);
    }
  };

  // fragment offsets: key 16 (r16 / 4) + 4 jt + r16 % 4, chunk 4 ks + g; value row 16 jd + r16, chunk 2 g + k2
  int koff[KS], voff[2];
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) {
    const int key = 16 * (r16 >> 2) + (r16 & 3);
    koff[ks] = key * (2 * D) + key_chunk<D>(key, 4 * ks + g) * 16;
  }
#pragma unroll
  for (int k2 = 0; k2 < 2; ++k2) voff[k2] = r16 * 128 + (((2 * g + k2) ^ (r16 & 7)) << 4);

  f32x4 o[RT][JD];
  float m[RT], l[RT];                                    // l: this lane's share of the row's sum
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int jd = 0; jd < JD; ++jd) o[i][jd] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  float vref = -INFINITY;

  uint32_t nan_out[RT];                                  // bit 4 jd + r: output d = 16 jd + 4 g + r is NaN
#pragma unroll
  for (int i = 0; i < RT; ++i) nan_out[i] = 0;
  auto compute = [&](int t, int buf, float kscale, float vscale, int have) {
    // some position of the block is masked for some row, absent, or in a page left out
    const bool edge = 64 * t + 64 > lo_lim || __any(have < 16);
    const int key0 = 64 * t + 16 * g;
    f32x4 sc[RT][4];
    // fragments of a key tile are read one tile ahead; the fences keep the
    // compiler from reading all of them at once, which spills
    const uint8_t* kr = smem[buf][0];
    half8 kf[2][KS];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) kf[0][ks] = *(const half8*)(kr + koff[ks]);
#pragma unroll
    for (int jt = 0; jt < 4; ++jt) {
      if (jt < 3) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) kf[(jt + 1) & 1][ks] = *(const half8*)(kr + koff[ks] + (jt + 1) * 8 * D);
      }
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int i = 0; i < RT; ++i)
          sc[i][jt] = mfma16(kf[jt & 1][ks], qf[i][ks], ks ? sc[i][jt] : f32x4{0.f, 0.f, 0.f, 0.f});
      __builtin_amdgcn_sched_barrier(0);
    }
    const float f = score_factor(kscale, a.scale_log2, have);
    if (edge) {
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const int seen = min(lim[i] - key0, have);       // of the lane's 16 positions
#pragma unroll
        for (int jt = 0; jt < 4; ++jt)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (4 * jt + r >= seen) sc[i][jt][r] = -INFINITY;
      }
    }
    const float lv = have > 0 ? __builtin_amdgcn_logf(vscale) : -INFINITY;
    f16x8 pf[RT][2];
    float sum[RT], rc;
    // w = 2^(s f + log2 c - m), c the lane's value scale over the reference; the
    // softmax's sum takes 1 / c once for the lane's 16 positions
    auto weights = [&]() {
      const float lc = scale_over(lv, vref, have);
      rc = __builtin_amdgcn_exp2f(-lc);
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        // a row that has seen nothing yet has m = -inf: its scores are all -inf
        const float ms = lc - (m[i] == -INFINITY ? 0.0f : m[i]);
        sum[i] = 0.f;
#pragma unroll
        for (int jt = 0; jt < 4; ++jt)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[i][jt][r], f, ms));
            sum[i] += w;
            pf[i][jt >> 1][4 * (jt & 1) + r] = (_Float16)w;
          }
      }
    };
    // The subtracted maximum and the value reference stay as they are while the
    // lane's weights sum to at most kMostSum (each is then within fp16): that is
    // asked after the fact, and only a block that exceeds it has its maximum
    // taken and its weights formed again.
    weights();
    bool grow = lv > vref + kLazyV;
#pragma unroll
    for (int i = 0; i < RT; ++i) grow = grow || m[i] == -INFINITY || sum[i] > kMostSum;
    if (__any(grow)) {
      const float lvm = max_over_g(lv), vn = lvm > vref + kLazyV ? lvm : vref;
      const float fv = vref == vn ? 1.0f : __builtin_amdgcn_exp2f(vref - vn);
      vref = vn;
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        float y = sc[i][0][0];
#pragma unroll
        for (int jt = 0; jt < 4; ++jt)
#pragma unroll
          for (int r = 0; r < 4; ++r) y = fmaxf(y, sc[i][jt][r]);
        const float mn = fmaxf(m[i], max_over_g(y * f));
        const float al = m[i] == mn ? 1.0f : __builtin_amdgcn_exp2f(m[i] - mn);
        l[i] *= al;
        m[i] = mn;
#pragma unroll
        for (int jd = 0; jd < JD; ++jd)
#pragma unroll
          for (int r = 0; r < 4; ++r) o[i][jd][r] *= al * fv;
      }
      weights();
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) l[i] += sum[i] * rc;
    const uint8_t* vt = smem[buf][1];
    auto vfrag = [&](int jd, int k2) { return *(const f16x8*)(vt + voff[k2] + jd * 2048); };
    f16x8 vf[2][2];                                      // likewise, of a d tile
    vf[0][0] = vfrag(0, 0);
    vf[0][1] = vfrag(0, 1);
#pragma unroll
    for (int jd = 0; jd < JD; ++jd) {
      if (jd + 1 < JD) {
        vf[(jd + 1) & 1][0] = vfrag(jd + 1, 0);
        vf[(jd + 1) & 1][1] = vfrag(jd + 1, 1);
      }
#pragma unroll
      for (int k2 = 0; k2 < 2; ++k2)
#pragma unroll
        for (int i = 0; i < RT; ++i) o[i][jd] = mfma16(vf[jd & 1][k2], pf[i][k2], o[i][jd]);
      __builtin_amdgcn_sched_barrier(0);
    }
    // Values that are not numbers were taken out of the block, since one row may
    // see what is masked for another: a row that sees one gets NaN. Row d = 16 jd
    // + .. was put by wave jd % NW.
    int put_by[NW], nans = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) nans |= put_by[w] = nan_of[buf][w];
    if (__builtin_amdgcn_readfirstlane(nans)) {
      uint64_t sees[RT];
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const int n = min(max(lim[i] - 64 * t, 0), 64);
        sees[i] = n == 64 ? ~0ull : (1ull << n) - 1;
      }
#pragma unroll
      for (int jd = 0; jd < JD; ++jd) {
        if (!__builtin_amdgcn_readfirstlane(put_by[jd % NW])) continue;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint64_t at = *(const uint64_t*)nan_at[buf][16 * jd + 4 * g + r];
#pragma unroll
          for (int i = 0; i < RT; ++i)
            nan_out[i] |= at & sees[i] ? 1u << (4 * jd + r) : 0u;
        }
      }
    }
  };

  if (tiles > 0) {
    load_ids(0);
    load(0);
    load_ids(1);
    put(0);
    float ks = nks, vs = nvs;
    int have = nhave;
    __syncthreads();
    for (int t = 0; t < tiles; ++t) {
      if (t + 1 < tiles) {
        load(t + 1);
        load_ids(t + 2);                                 // clamped to the last positions
      }
      // a block that none of the wave's rows sees is passed over; the barrier is not
      if (64 * t < hi_lim) {
        compute(t, t & 1, ks, vs, have);
      }
      if (t + 1 < tiles) {
        put((t + 1) & 1);
        ks = nks;
        vs = nvs;
        have = nhave;
      }
      __syncthreads();
    }
  }

  const float vscale = vref == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(vref);
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    float ll = l[i];
    ll += __shfl_xor(ll, 16);
    ll += __shfl_xor(ll, 32);
    const int row = wave_base + 16 * i + r16;
    if (row >= rows) continue;
    const float inv = ll == 0.f ? 0.0f : vscale / ll;
    const int tok = row / a.group, hh = row - tok * a.group;
    uint16_t* op = a.out + (s.c0 + tok) * a.ldo + (int64_t)(h * a.group + hh) * D + 4 * g;
#pragma unroll
    for (int jd = 0; jd < JD; ++jd) {
      float v[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = nan_out[i] >> (4 * jd + r) & 1 ? NAN : o[i][jd][r] * inv;
      *(uint2*)(op + 16 * jd) = make_uint2(pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]));
    }
  }
}

// Joins the parts of a split sequence: a wave for each (row, head). Parts past a
// row's limit have m = -inf, l = 0.
template <int DT, int D>
__global__ __launch_bounds__(256) void k_kv_join(const AttnArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int b = blockIdx.x, h = blockIdx.y;
  const int64_t run = run_length(a, tiles_before(a, a.batch)), before = tiles_before(a, b);
  const int first = (int)(before / run), parts = (int)((before + tiles_of(a, b) - 1) / run) - first + 1;
  if (parts <= 1) return;
  const Seq s = seq_of(a, b);
  const int rows = s.n * a.group;
  for (int row = blockIdx.z * 4 + wave; row < rows; row += gridDim.z * 4) {
    const int64_t at0 = ((int64_t)(first + b) * a.hk + h) * a.max_rows + row, step = (int64_t)a.hk * a.max_rows;
    float mm = -INFINITY;
    for (int i = lane; i < parts; i += 64) {
      const f32x2 ml = *(const f32x2*)(a.part_ml + (at0 + i * step) * 2);
      if (ml[1] != 0.f) mm = fmaxf(mm, ml[0]);
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) mm = fmaxf(mm, __shfl_xor(mm, o));
    float ll = 0.f;
    f32x2 acc{0.f, 0.f};
#pragma unroll 8
    for (int i = 0; i < parts; ++i) {
      const int64_t at = at0 + i * step;
      const f32x2 ml = *(const f32x2*)(a.part_ml + at * 2);
      f32x2 v{0.f, 0.f};
      if constexpr (D == 128) v = *(const f32x2*)(a.part_o + at * D + 2 * lane);
      else v[0] = a.part_o[at * D + lane];
      const bool some = ml[1] != 0.f;                    // NaN counts
      const float f = some ? __builtin_amdgcn_exp2f(ml[0] - mm) : 0.f;
      ll += some ? ml[1] * f : 0.f;
      acc[0] += some ? v[0] * f : 0.f;
      acc[1] += some ? v[1] * f : 0.f;
    }
    const float inv = ll == 0.f ? 0.0f : 1.0f / ll;
    const int tok = row / a.group, hh = row - tok * a.group;
    uint16_t* op = a.out + (s.c0 + tok) * a.ldo + (int64_t)(h * a.group + hh) * D;
    if constexpr (D == 128) *(uint32_t*)(op + 2 * lane) = pack2<DT>(acc[0] * inv, acc[1] * inv);
    else op[lane] = (uint16_t)pack2<DT>(acc[0] * inv, 0.f);
  }
}

// ---------------------------------------------------------------------------
// Launchers
// ---------------------------------------------------------------------------
template <int DT>
void launch_append(const AppendArgs& a, int64_t batch, hipStream_t st) {
  LaunchTimer t("kv_append", st);
  const dim3 grid((unsigned)((a.max_new + a.page - 2) / a.page + 1), (unsigned)batch, (unsigned)(2 * a.heads));
  const int most = a.page < a.max_new ? a.page : (int)a.max_new;       // new tokens of one block
  const size_t lds = (size_t)a.d * (a.page + 4);
  // one wave where a block's new tokens fit it (single tokens): more blocks in
  // flight, no barriers; 256 threads otherwise
  if (most * a.d / 8 <= 64) QAT_LAUNCH((k_kv_append<DT, 64, 1>), grid, dim3(64), lds, st, a);
  else if (most * a.d / 8 <= 512) QAT_LAUNCH((k_kv_append<DT, 256, 2>), grid, dim3(256), lds, st, a);
  else if (most * a.d / 8 <= 1024) QAT_LAUNCH((k_kv_append<DT, 256, 4>), grid, dim3(256), lds, st, a);
  else QAT_LAUNCH((k_kv_append<DT, 256, 8>), grid, dim3(256), lds, st, a);
}

struct AttnPlan {
  bool prompt;                     // the prompts' kernel
  int row_blocks, target, parts;
  size_t ml_at, bytes;             // workspace: part_o, then part_ml
};

constexpr int kTargetGroups = 256; // one workgroup for each CU: two measured the same on long caches, slower on short ones

AttnPlan plan_attn(int64_t batch, int64_t hk, int64_t group, int d, int64_t max_new, int64_t max_len) {
  AttnPlan p;
  const int64_t rows = max_new * group;
  // Prompts' kernel or the other one by how many workgroups the first would have.
  // It does not split a sequence, and a workgroup takes 1.7 us a block of
  // positions however few there are (1 x 20 tokens over 8000, 8 key heads, 8
  // workgroups: 217 us, the other kernel 27; 1 x 300 over 4000, 80: 114 and 70;
  // 1 x 700 over 2000, 176: 61 and 66; 2 x 2048 over themselves, 1024: 92 and 170).
  p.prompt = rows > 32 && batch * hk * ((rows + 127) / 128) * 4 >= 3 * kTargetGroups;
  if (p.prompt) {
    p.row_blocks = (int)((rows + 127) / 128);
    p.target = p.parts = 0;
    p.ml_at = p.bytes = 0;
    return p;
  }
  p.row_blocks = (int)((rows + 15) / 16);
  const int64_t per = hk * p.row_blocks;
  const bool split = max_len > kMinTiles * kTile && per < kTargetGroups;
  p.target = split ? (int)((kTargetGroups + per - 1) / per) : 0;
  p.parts = (int)(batch + p.target);         // at most
  p.ml_at = p.bytes = 0;
  if (split) {
    const int64_t n = (int64_t)p.parts * hk * rows;
    p.ml_at = (size_t)((n * d * 4 + 255) / 256 * 256);
    p.bytes = p.ml_at + (size_t)((n * 8 + 255) / 256 * 256);
  }
  return p;
}

template <int DT, int D>
void launch_attn(const AttnArgs& a, const AttnPlan& p, hipStream_t st) {
  if (p.prompt) {
    LaunchTimer t("kv_attn", st);
    const dim3 grid((unsigned)((int64_t)p.row_blocks * a.batch * a.hk));
    QAT_LAUNCH((k_kv_prompt<DT, D>), grid, dim3(256), 0, st, a);
    return;
  }
  {
    LaunchTimer t("kv_attn", st);
    const dim3 grid((unsigned)(a.target ? a.target : a.batch), (unsigned)a.hk, (unsigned)p.row_blocks);
    QAT_LAUNCH((k_kv_decode<DT, D>), grid, dim3(256), 0, st, a);
  }
  if (a.target) {
    LaunchTimer t("kv_attn_join", st);
    const int z = (a.max_rows + 3) / 4;
    QAT_LAUNCH((k_kv_join<DT, D>), dim3((unsigned)a.batch, (unsigned)a.hk, (unsigned)(z < 64 ? z : 64)), dim3(256),
               0, st, a);
  }
}

int log2_page(int32_t page) { return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : page == 128 ? 7 : -1; }

constexpr int64_t kMaxGrid = 65535;          // of a launch's y and z

int32_t check_batch(int32_t dtype, int64_t tokens, int64_t batch, int32_t heads, int32_t d, int64_t cols,
                    int32_t page, int64_t n_pages, int64_t max_new) {
  if (dtype != QAT_BF16 && dtype != QAT_F16) return QAT_ERR_TYPE;
  if (d != 64 && d != 128) return QAT_ERR_SHAPE;
  if (log2_page(page) < 0) return QAT_ERR_SHAPE;
  if (tokens < 0 || batch < 0 || heads <= 0 || cols <= 0 || n_pages <= 0 || max_new < 0) return QAT_ERR_SHAPE;
  if (tokens > kMaxCount || batch > kMaxGrid || heads > 1024 || cols * page > kMaxCount || n_pages > kMaxCount ||
      max_new > kMaxCount || n_pages * heads >= (int64_t(1) << 31))
    return QAT_ERR_SHAPE;
  return QAT_OK;
}

int32_t check_ld(int64_t ld, int64_t row) {
  if (ld < row || ld > kMaxCount) return QAT_ERR_SHAPE;
  return ld % 8 ? QAT_ERR_ALIGN : QAT_OK;
}

}  // namespace
}  // namespace qat

QAT_API int32_t qat_rope_inv_freq(int32_t rot, double base, int32_t scaling, double factor, int64_t original,
                                  double beta_fast, double beta_slow, float* inv_freq, float* mscale) {
  if (!inv_freq || !mscale) return QAT_ERR_NULL;
  if (scaling < QAT_ROPE_PLAIN || scaling > QAT_ROPE_PARTS) return QAT_ERR_TYPE;
  if (rot < 2 || rot % 2 || !(base > 1) || !(base < 1e300)) return QAT_ERR_SHAPE;
  if (scaling != QAT_ROPE_PLAIN && !(factor >= 1 && factor < 1e9)) return QAT_ERR_SHAPE;
  const bool parts = scaling == QAT_ROPE_PARTS;
  if (parts && (original <= 0 || !(beta_slow > 0) || !(beta_fast > beta_slow) || !(beta_fast < 1e9)))
    return QAT_ERR_SHAPE;
  // the pair index that turns `turns` times over the original context
  auto pair_of = [&](double turns) { return rot * log((double)original / (turns * 2 * M_PI)) / (2 * log(base)); };
  double lo = 0, hi = 0;
  if (parts) {
    lo = fmax(floor(pair_of(beta_fast)), 0);
    hi = fmin(ceil(pair_of(beta_slow)), rot - 1);
    if (hi <= lo) hi = lo + 0.001;
  }
  for (int i = 0; i < rot / 2; ++i) {
    double f = pow(base, -2.0 * i / rot);
    if (scaling == QAT_ROPE_LINEAR) f /= factor;
    if (parts) {
      const double w = 1 - fmin(fmax((i - lo) / (hi - lo), 0), 1);
      f = f * (1 - w) / factor + f * w;
    }
    inv_freq[i] = (float)f;
  }
  *mscale = parts && factor > 1 ? (float)(0.1 * log(factor) + 1) : 1.0f;
  return QAT_OK;
}

QAT_API int32_t qat_rope(const void* q, const void* k, const int32_t* pos, const float* inv_freq, int64_t tokens,
                         int32_t heads_q, int32_t heads_k, int32_t head_dim, int32_t rot, int32_t half,
                         int32_t inverse, float mscale, int32_t dtype, int64_t ldq, int64_t ldk, void* q_out,
                         int64_t ldq_out, void* k_out, int64_t ldk_out, hipStream_t stream) {
  using namespace qat;
  if (dtype != QAT_BF16 && dtype != QAT_F16) return QAT_ERR_TYPE;
  if ((half != 0 && half != 1) || (inverse != 0 && inverse != 1)) return QAT_ERR_TYPE;
  if (tokens < 0 || tokens > kMaxCount || heads_q <= 0 || heads_q > 4096 || heads_k < 0 || heads_k > 4096 ||
      (head_dim != 64 && head_dim != 128) || rot < 16 || rot > head_dim || rot % 16)
    return QAT_ERR_SHAPE;
  const int64_t rq = (int64_t)heads_q * head_dim, rk = (int64_t)heads_k * head_dim;
  QAT_CHECK(check_ld(ldq, rq));
  QAT_CHECK(check_ld(ldq_out, rq));
  if (heads_k) {
    QAT_CHECK(check_ld(ldk, rk));
    QAT_CHECK(check_ld(ldk_out, rk));
  }
  if (tokens == 0) return QAT_OK;
  QAT_CHECK(check_required({q, pos, inv_freq, q_out}));
  if (heads_k ? (!k || !k_out) : (k || k_out)) return QAT_ERR_NULL;
  QAT_CHECK(check_aligned({q, k, q_out, k_out}));
  if (((uintptr_t)pos | (uintptr_t)inv_freq) & 3) return QAT_ERR_ALIGN;
  const Span sq{q, strided_bytes(tokens, ldq, rq, 2)}, sk{k, strided_bytes(tokens, ldk, rk, 2)};
  const Span oq{q_out, strided_bytes(tokens, ldq_out, rq, 2)}, ok{k_out, strided_bytes(tokens, ldk_out, rk, 2)};
  const bool in_q = q == q_out && ldq == ldq_out, in_k = k && k == k_out && ldk == ldk_out;
  const Span sp{pos, (size_t)tokens * 4}, sf{inv_freq, (size_t)rot * 2};
  QAT_CHECK(check_spans({oq}, {sp, sf}));
  QAT_CHECK(check_spans({ok}, {sp, sf}));
  // q and k may be slices of one packed projection
  if (!in_q) QAT_CHECK(check_rows_apart(oq, ldq_out, rq, sq, ldq, rq));
  if (heads_k) {
    if (!in_k) QAT_CHECK(check_rows_apart(ok, ldk_out, rk, sk, ldk, rk));
    QAT_CHECK(check_rows_apart(oq, ldq_out, rq, sk, ldk, rk));
    QAT_CHECK(check_rows_apart(ok, ldk_out, rk, sq, ldq, rq));
    QAT_CHECK(check_rows_apart(oq, ldq_out, rq, ok, ldk_out, rk));
  }
  RopeArgs a;
  a.q = (const uint16_t*)q;
  a.k = (const uint16_t*)k;
  a.qo = (uint16_t*)q_out;
  a.ko = (uint16_t*)k_out;
  a.pos = pos;
  a.inv_freq = inv_freq;
  a.ldq = ldq;
  a.ldk = ldk;
  a.ldqo = ldq_out;
  a.ldko = ldk_out;
  a.hq = heads_q;
  a.hk = heads_k;
  a.d = head_dim;
  a.rot = rot;
  a.half = half;
  a.pieces = head_dim / 16;
  a.mscale = mscale;
  a.sign = inverse ? -1.0f : 1.0f;
  // few tokens: a token's heads over several workgroups, so that each thread has one piece
  const int need = (int)(((int64_t)(heads_q + heads_k) * a.pieces + 255) / 256);
  const int split = tokens < 256 ? need : 1;
  LaunchTimer t("rope", stream);
  const dim3 grid((unsigned)tokens, (unsigned)split);
  if (dtype == QAT_BF16) QAT_LAUNCH(k_rope<QAT_BF16>, grid, dim3(256), 0, stream, a);
  else QAT_LAUNCH(k_rope<QAT_F16>, grid, dim3(256), 0, stream, a);
  return finish_call();
}

QAT_API int32_t qat_kv_append(const void* k, const void* v, int32_t dtype, int64_t ldk, int64_t ldv,
                              const int32_t* cu, const int32_t* lens, const int32_t* table, int64_t table_cols,
                              int64_t tokens, int64_t batch, int32_t heads, int32_t head_dim, int32_t page,
                              int64_t n_pages, int64_t max_new, uint8_t* k_cache, uint8_t* v_cache, float* k_scale,
                              float* v_scale, hipStream_t stream) {
  using namespace qat;
  QAT_CHECK(check_batch(dtype, tokens, batch, heads, head_dim, table_cols, page, n_pages, max_new));
  const int64_t row = (int64_t)heads * head_dim;
  QAT_CHECK(check_ld(ldk, row));
  QAT_CHECK(check_ld(ldv, row));
  if (tokens == 0 || batch == 0 || max_new == 0) return QAT_OK;
  QAT_CHECK(check_required({k, v, cu, lens, table, k_cache, v_cache, k_scale, v_scale}));
  QAT_CHECK(check_aligned({k, v, k_cache, v_cache}));
  if (((uintptr_t)cu | (uintptr_t)lens | (uintptr_t)table | (uintptr_t)k_scale | (uintptr_t)v_scale) & 3)
    return QAT_ERR_ALIGN;
  const size_t nc = (size_t)(n_pages * row * page), ns = (size_t)(n_pages * heads * 4);
  QAT_CHECK(check_spans({{k_cache, nc}, {v_cache, nc}, {k_scale, ns}, {v_scale, ns}},
                        {{k, strided_bytes(tokens, ldk, row, 2)}, {v, strided_bytes(tokens, ldv, row, 2)},
                         {cu, (size_t)(batch + 1) * 4}, {lens, (size_t)batch * 4},
                         {table, (size_t)(batch * table_cols) * 4}}));
  AppendArgs a;
  a.x[0] = (const uint16_t*)k;
  a.x[1] = (const uint16_t*)v;
  a.ld[0] = ldk;
  a.ld[1] = ldv;
  a.cache[0] = k_cache;
  a.cache[1] = v_cache;
  a.scale[0] = k_scale;
  a.scale[1] = v_scale;
  a.cu = cu;
  a.lens = lens;
  a.table = table;
  a.cols = table_cols;
  a.tokens = tokens;
  a.n_pages = n_pages;
  a.max_new = max_new < tokens ? max_new : tokens;
  a.heads = heads;
  a.d = head_dim;
  a.page = page;
  if (dtype == QAT_BF16) launch_append<QAT_BF16>(a, batch, stream);
  else launch_append<QAT_F16>(a, batch, stream);
  return finish_call();
}

QAT_API size_t qat_kv_attn_ws_bytes(int64_t tokens, int64_t batch, int32_t heads_q, int32_t heads_kv,
                                    int32_t head_dim, int64_t max_new, int64_t max_len) {
  using namespace qat;
  if (heads_q <= 0 || heads_kv <= 0 || heads_q % heads_kv || max_len < 0 || max_len > kMaxCount ||
      check_batch(QAT_BF16, tokens, batch, heads_kv, head_dim, 1, 16, 1, max_new) != QAT_OK)
    return 0;
  const int64_t mn = max_new < tokens ? max_new : tokens;
  if (mn == 0 || batch == 0) return 0;
  return plan_attn(batch, heads_kv, heads_q / heads_kv, head_dim, mn, max_len).bytes;
}

QAT_API int32_t qat_kv_attn(const void* q, int32_t dtype, int64_t ldq, const int32_t* cu, const int32_t* lens,
                            const int32_t* table, int64_t table_cols, int64_t tokens, int64_t batch,
                            int32_t heads_q, int32_t heads_kv, int32_t head_dim, int32_t page, int64_t n_pages,
                            const uint8_t* k_cache, const uint8_t* v_cache, const float* k_scale,
                            const float* v_scale, float softmax_scale, int32_t causal, int64_t max_new,
                            int64_t max_len, void* out, int64_t ldo, void* ws, size_t ws_bytes, hipStream_t stream) {
  using namespace qat;
  QAT_CHECK(check_batch(dtype, tokens, batch, heads_kv, head_dim, table_cols, page, n_pages, max_new));
  if (causal != 0 && causal != 1) return QAT_ERR_TYPE;
  if (heads_q <= 0 || heads_q > 4096 || heads_q % heads_kv || max_len < 0 || max_len > kMaxCount ||
      !(softmax_scale > 0) || !(softmax_scale < INFINITY))
    return QAT_ERR_SHAPE;
  if ((max_new < tokens ? max_new : tokens) * (heads_q / heads_kv) > kMaxCount) return QAT_ERR_SHAPE;
  const int64_t row = (int64_t)heads_q * head_dim, krow = (int64_t)heads_kv * head_dim;
  QAT_CHECK(check_ld(ldq, row));
  QAT_CHECK(check_ld(ldo, row));
  const int64_t mn = max_new < tokens ? max_new : tokens;
  if (mn == 0 || batch == 0) return QAT_OK;
  QAT_CHECK(check_required({q, cu, lens, table, k_cache, v_cache, k_scale, v_scale, out}));
  QAT_CHECK(check_aligned({q, k_cache, v_cache, out, ws}));
  if (((uintptr_t)cu | (uintptr_t)lens | (uintptr_t)table | (uintptr_t)k_scale | (uintptr_t)v_scale) & 3)
    return QAT_ERR_ALIGN;
  const AttnPlan p = plan_attn(batch, heads_kv, heads_q / heads_kv, head_dim, mn, max_len);
  // grids: rows of a few sequences along z, of prompts with sequences and heads along x
  if (p.prompt ? (int64_t)p.row_blocks * batch * heads_kv > 0x7FFFFFFF : p.row_blocks > kMaxGrid) return QAT_ERR_SHAPE;
  if (p.bytes && (!ws || ws_bytes < p.bytes)) return QAT_ERR_WORKSPACE;
  const size_t nc = (size_t)(n_pages * krow * page), ns = (size_t)(n_pages * heads_kv * 4);
  QAT_CHECK(check_spans({{out, strided_bytes(tokens, ldo, row, 2)}, {ws, p.bytes}},
                        {{q, strided_bytes(tokens, ldq, row, 2)}, {k_cache, nc}, {v_cache, nc}, {k_scale, ns},
                         {v_scale, ns}, {cu, (size_t)(batch + 1) * 4}, {lens, (size_t)batch * 4},
                         {table, (size_t)(batch * table_cols) * 4}}));
  AttnArgs a;
  a.q = (const uint16_t*)q;
  a.ldq = ldq;
  a.cu = cu;
  a.lens = lens;
  a.table = table;
  a.cols = table_cols;
  a.tokens = tokens;
  a.n_pages = n_pages;
  a.batch = (int)batch;
  a.hk = heads_kv;
  a.group = heads_q / heads_kv;
  a.log_page = log2_page(page);
  a.k = k_cache;
  a.v = v_cache;
  a.ks = k_scale;
  a.vs = v_scale;
  a.scale_log2 = softmax_scale * 1.4426950408889634f;
  a.causal = causal;
  a.max_new = mn;
  a.max_len = max_len;
  a.out = (uint16_t*)out;
  a.ldo = ldo;
  a.target = p.target;
  a.max_rows = (int)(mn * a.group);
  a.row_blocks = p.row_blocks;
  a.part_o = (float*)ws;
  a.part_ml = (float*)((uint8_t*)ws + p.ml_at);
  if (head_dim == 128) {
    if (dtype == QAT_BF16) launch_attn<QAT_BF16, 128>(a, p, stream);
    else launch_attn<QAT_F16, 128>(a, p, stream);
  } else {
    if (dtype == QAT_BF16) launch_attn<QAT_BF16, 64>(a, p, stream);
    else launch_attn<QAT_F16, 64>(a, p, stream);
  }
  return finish_call();
}
