// Microscaled 4-bit floating point (MXFP4): quantisation and the product on
// the block-scaled matrix instructions (gfx950, wave64).
//
// Format: 32 consecutive elements of a row share the scale 2^e (byte e + 127);
// elements are E2M1 codes, two to a byte, the even element in the low half.
#include <type_traits>

#include "../../include/qat_mx.h"
#include "qat_check.h"
#include "qat_device.h"
#include "qat_dma.h"
#include "qat_internal.h"

namespace qat {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

// ---------------------------------------------------------------------------
// Quantisation. A thread owns 8 consecutive elements, four lanes a block: the
// block's largest magnitude is the largest of the elements' fp32 bits without
// the sign (integers order like magnitudes, and infinities and NaN come out on
// top), joined over the four lanes by two DPP exchanges. x 2^-e is exact, so
// the only rounding is the conversion's own. One pass over X; bound by HBM: 11008
// x 4096 fp32 with codes, scales and values in 70 us, 5.5 TB/s.
// ---------------------------------------------------------------------------
template <int DT>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&x)[8]) {
  if constexpr (DT == QAT_F32) {
    const f32x4 a = *(const f32x4*)((const float*)p + i), b = *(const f32x4*)((const float*)p + i + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[j] = a[j];
      x[j + 4] = b[j];
    }
  } else if constexpr (DT == QAT_BF16) {
    const uint4 v = *(const uint4*)((const uint16_t*)p + i);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = __builtin_bit_cast(float, w[j] << 16);
      x[2 * j + 1] = __builtin_bit_cast(float, w[j] & 0xFFFF0000u);
    }
  } else {
    typedef _Float16 f16x8_ __attribute__((ext_vector_type(8)));
    const f16x8_ v = *(const f16x8_*)((const _Float16*)p + i);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = (float)v[j];
  }
}

__device__ __forceinline__ uint32_t pack2(float a, float b, int dtype) {
  if (dtype == QAT_BF16) return pack_bf16x2(a, b);
  return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b});
}

template <int DT>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&x)[8]) {
  if constexpr (DT == QAT_F32) {
    *(f32x4*)((float*)p + i) = f32x4{x[0], x[1], x[2], x[3]};
    *(f32x4*)((float*)p + i + 4) = f32x4{x[4], x[5], x[6], x[7]};
  } else {
    *(uint4*)((uint16_t*)p + i) = make_uint4(pack2(x[0], x[1], DT), pack2(x[2], x[3], DT), pack2(x[4], x[5], DT),
                                             pack2(x[6], x[7], DT));
  }
}

template <int kCtrl>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, kCtrl, 0xF, 0xF, false);
}

// The lane's 8 codes (a dword) and its block's scale byte; every lane of the
// block's four calls it together.
__device__ __forceinline__ uint32_t quant8(const float (&x)[8], uint32_t& byte) {
  uint32_t a = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) a = max(a, __builtin_bit_cast(uint32_t, x[j]) & 0x7FFFFFFFu);
  a = max(a, dpp_u32<kDppXor1>(a));
  a = max(a, dpp_u32<kDppXor2>(a));
  const bool odd = a >= 0x7F800000u;
  const uint32_t ex = a >> 23;
  byte = odd ? 255u : (ex > 2 ? ex - 2 : 0u);
  // 2^-e = 2^(127 - byte), a normal number for every byte up to 252
  const float inv = __builtin_bit_cast(float, odd ? 0u : (254u - byte) << 23);
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[0] * inv, x[1] * inv, 1.0f, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[2] * inv, x[3] * inv, 1.0f, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[4] * inv, x[5] * inv, 1.0f, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[6] * inv, x[7] * inv, 1.0f, 3);
  return odd ? 0u : c;
}

struct QuantArgs {
  const void* X;
  int64_t ldx;
  uint32_t chunks;      // rows * cols / 8, below 2^31
  uint32_t row_chunks;  // cols / 8
  FastDiv div;          // by row_chunks
  uint8_t* codes;
  uint8_t* scales;
  void* x_hat;
};

template <int DT>
__global__ __launch_bounds__(256) void k_mx_quant(const QuantArgs a) {
  // chunks is a multiple of 4, so the four lanes of a block are all in or out
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  if (i >= a.chunks) return;
  const uint32_t row = a.div.div(i), col = (i - row * a.row_chunks) * 8;
  float x[8];
  load8<DT>(a.X, (int64_t)row * a.ldx + col, x);
  uint32_t byte;
  const uint32_t c = quant8(x, byte);
  if (a.codes) {
    *(uint32_t*)(a.codes + (int64_t)i * 4) = c;
    if ((i & 3) == 0) a.scales[i >> 2] = (uint8_t)byte;
  }
  if (a.x_hat) {
    // 2^e; the byte 0 is 2^-127, a subnormal, and 255 an infinity that makes
    // NaN of the zero codes
    const float s = __builtin_bit_cast(float, byte ? byte << 23 : 0x00400000u);
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f32x2 p;
      if (j == 0) p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0);
      else if (j == 1) p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1);
      else if (j == 2) p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2);
      else p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3);
      v[2 * j] = p[0] * s;
      v[2 * j + 1] = p[1] * s;
    }
    store8<DT>(a.x_hat, (int64_t)i * 8, v);
  }
}

// ---------------------------------------------------------------------------
// Product, v_mfma_scale_f32_16x16x128_f8f6f4 with both operands E2M1: lane l
// holds 32 consecutive elements (16 bytes) of row l & 15 and their scale.
// The contraction's order is free as long as both operands share it: over 512
// elements (16 blocks) lane group g = l >> 4 takes block 4 g + j in step j, so
// a lane reads 64 consecutive bytes of its row and its four scales are one
// dword, whose byte j the instruction selects.
// ---------------------------------------------------------------------------
struct Piece {
  i32x4 c[4];
  uint32_t s;
};

struct ProductArgs {
  const uint8_t* xc;
  const uint8_t* xs;
  const uint8_t* wc;
  const uint8_t* ws;
  int M, N, K;
  void* Y;
  int64_t ldy;
  const void* x16;                 // X in 16 bits, quantised by the product itself
  int64_t ldx;
};

// Superstep ss of a row: blocks 16 ss + 4 g .. + 3, those past the row's end zero.
__device__ __forceinline__ void load_piece(Piece& p, const uint8_t* codes, const uint8_t* scales, int nblk, int ss,
                                           int g) {
  const int b0 = 16 * ss + 4 * g;
  if (b0 + 4 <= nblk) {
#pragma unroll
    for (int j = 0; j < 4; ++j) p.c[j] = *(const i32x4*)(codes + (int64_t)(b0 + j) * 16);
    __builtin_memcpy(&p.s, scales + b0, 4);
  } else {
    p.s = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      p.c[j] = i32x4{0, 0, 0, 0};
      if (b0 + j < nblk) {
        p.c[j] = *(const i32x4*)(codes + (int64_t)(b0 + j) * 16);
        p.s |= (uint32_t)scales[b0 + j] << (8 * j);
      }
    }
  }
}

__device__ __forceinline__ i32x8 wide(i32x4 v) { return i32x8{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }

__device__ __forceinline__ f32x4 mfma4(const Piece& a, const Piece& b, f32x4 acc) {
  acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(a.c[0]), wide(b.c[0]), acc, 4, 4, 0, a.s, 0, b.s);
  acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(a.c[1]), wide(b.c[1]), acc, 4, 4, 1, a.s, 1, b.s);
  acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(a.c[2]), wide(b.c[2]), acc, 4, 4, 2, a.s, 2, b.s);
  acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(a.c[3]), wide(b.c[3]), acc, 4, 4, 3, a.s, 3, b.s);
  return acc;
}

// Four consecutive outputs n .. n + 3 of one token.
template <int DT>
__device__ __forceinline__ void store_out(void* Y, int64_t ldy, int m, int n, int N, f32x4 v) {
  uint16_t* y = (uint16_t*)Y + (int64_t)m * ldy + n;
  const uint32_t lo = pack2(v[0], v[1], DT), hi = pack2(v[2], v[3], DT);
  if (n + 4 <= N && ((uintptr_t)y & 7) == 0) {
    *(uint2*)y = make_uint2(lo, hi);
  } else {
    if (n < N) y[0] = (uint16_t)lo;
    if (n + 1 < N) y[1] = (uint16_t)(lo >> 16);
    if (n + 2 < N) y[2] = (uint16_t)hi;
    if (n + 3 < N) y[3] = (uint16_t)(hi >> 16);
  }
}

// Eight of them.
template <int DT>
__device__ __forceinline__ void store_out8(void* Y, int64_t ldy, int m, int n, int N, f32x4 v, f32x4 w) {
  uint16_t* y = (uint16_t*)Y + (int64_t)m * ldy + n;
  if (n + 8 <= N && ((uintptr_t)y & 15) == 0) {
    *(uint4*)y = make_uint4(pack2(v[0], v[1], DT), pack2(v[2], v[3], DT), pack2(w[0], w[1], DT), pack2(w[2], w[3], DT));
  } else {
    store_out<DT>(Y, ldy, m, n, N, v);
    store_out<DT>(Y, ldy, m, n + 4, N, w);
  }
}

// Few tokens: a workgroup owns 16 weight rows and 16 tokens; its 8 waves split
// the contraction by supersteps and meet in LDS. Bound by the weights' bytes and,
// at these sizes, by latency: 1 x 4096 -> 11008 in 6.6 us, 3.6 TB/s.
//
// kQuant: X comes in 16 bits and is quantised here, one launch for the linear
// layer of a served token. A wave quantises its own supersteps (8 elements a
// lane, a token at a time) while its weights arrive, and turns them into the
// operand's order through its own LDS. Every workgroup does so again, which pays
// for up to kQuantTokens tokens.
constexpr int kQuantTokens = 4;

template <int DT, bool kQuant>
__global__ __launch_bounds__(512) void k_mx_skinny(const ProductArgs a) {
  __shared__ f32x4 part[8][64];
  // codes and scales of a superstep
  __shared__ __attribute__((aligned(16))) uint8_t xq[kQuant ? 8 : 1][kQuant ? kQuantTokens : 1][272];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r16 = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * 16, m0 = blockIdx.y * 16;
  const int nblk = a.K / 32, nss = (nblk + 15) / 16;
  const int64_t wr = min(n0 + r16, a.N - 1), xr = min(m0 + r16, a.M - 1);
  const uint8_t* wc = a.wc + wr * (a.K / 2);
  const uint8_t* ws = a.ws + wr * nblk;
  f32x4 acc{0.f, 0.f, 0.f, 0.f};
  for (int ss = wave; ss < nss; ss += 8) {
    Piece w, x;
    load_piece(w, wc, ws, nblk, ss, g);
    if constexpr (kQuant) {
      const int col = ss * 512 + 8 * lane;
      for (int m = 0; m < a.M; ++m) {
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (col < a.K) load8<DT>(a.x16, m * a.ldx + col, v);       // the same for a block's four lanes
        uint32_t byte;
        *(uint32_t*)&xq[wave][m][4 * lane] = quant8(v, byte);
        if ((lane & 3) == 0) xq[wave][m][256 + (lane >> 2)] = (uint8_t)byte;
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int j = 0; j < 4; ++j) x.c[j] = *(const i32x4*)&xq[wave][xr][64 * g + 16 * j];
      x.s = *(const uint32_t*)&xq[wave][xr][256 + 4 * g];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    } else {
      load_piece(x, a.xc + xr * (a.K / 2), a.xs + xr * nblk, nblk, ss, g);
    }
    acc = mfma4(w, x, acc);
  }
  part[wave][lane] = acc;
  __syncthreads();
  if (threadIdx.x < 64) {
#pragma unroll
    for (int w = 1; w < 8; ++w) acc += part[w][lane];
    if (m0 + r16 < a.M) store_out<DT>(a.Y, a.ldy, m0 + r16, n0 + 4 * g, a.N, acc);
  }
}

// ---------------------------------------------------------------------------
// Scales in the order of the tiled product: for each row and 512 elements (16
// blocks, the last ones zero past the row's end) the bytes [g][j] of blocks
// 4 j + g, so that lane group g has the scales of four steps in one dword.
// What the zero scales (2^-127, of both operands) multiply is below 2^-245 and
// vanishes, so codes past a row's end need no masking. One thread transposes
// 16 bytes; a few microseconds beside the product, whose inner loop it frees of
// byte reads, alignment and the ragged end.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint4 transpose4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  // __builtin_amdgcn_perm(hi, lo, selector): bytes 0-3 of lo, 4-7 of hi
  const uint32_t ab0 = __builtin_amdgcn_perm(b, a, 0x05010400u), ab1 = __builtin_amdgcn_perm(b, a, 0x07030602u);
  const uint32_t cd0 = __builtin_amdgcn_perm(d, c, 0x05010400u), cd1 = __builtin_amdgcn_perm(d, c, 0x07030602u);
  return make_uint4(__builtin_amdgcn_perm(cd0, ab0, 0x05040100u), __builtin_amdgcn_perm(cd0, ab0, 0x07060302u),
                    __builtin_amdgcn_perm(cd1, ab1, 0x05040100u), __builtin_amdgcn_perm(cd1, ab1, 0x07060302u));
}

struct ReorderArgs {
  const uint8_t* src[2];           // X's scales, W's
  uint8_t* dst[2];
  int64_t n0, n1;                  // 16-byte pieces of each
  int nblk, nss;
};

// 16-byte piece i of one operand.
__device__ __forceinline__ void reorder_piece(const uint8_t* src, uint8_t* dst, int64_t i, int nblk, int nss) {
  const int64_t row = i / nss;
  const int b0 = (int)(i - row * nss) * 16, n = min(nblk - b0, 16);
  const uint8_t* p = src + row * nblk + b0;
  uint32_t w[4] = {0, 0, 0, 0};
  if (n == 16) {
    __builtin_memcpy(w, p, 16);
  } else {
#pragma unroll
    for (int k = 0; k < 16; ++k)
      if (k < n) w[k >> 2] |= (uint32_t)p[k] << (8 * (k & 3));
  }
  *(uint4*)(dst + i * 16) = transpose4(w[0], w[1], w[2], w[3]);
}

__global__ __launch_bounds__(256) void k_mx_reorder(const ReorderArgs a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < a.n0) reorder_piece(a.src[0], a.dst[0], i, a.nblk, a.nss);
  else if (i < a.n0 + a.n1) reorder_piece(a.src[1], a.dst[1], i - a.n0, a.nblk, a.nss);
}

// qat_mx_linear before the tiled product, one launch: the first x_blocks
// workgroups quantise X and write its scales in the tiled order (a thread has 8
// elements, rows padded to 512), the others reorder W's.
struct PrepareArgs {
  const void* X;
  int64_t ldx, x_chunks;           // rows * nss * 64
  int x_blocks, cols;
  uint8_t* codes;
  ReorderArgs r;
};

template <int DT>
__global__ __launch_bounds__(256) void k_mx_prepare(const PrepareArgs a) {
  if ((int)blockIdx.x >= a.x_blocks) {
    const int64_t i = (int64_t)((int)blockIdx.x - a.x_blocks) * 256 + threadIdx.x;
    if (i < a.r.n1) reorder_piece(a.r.src[1], a.r.dst[1], i, a.r.nblk, a.r.nss);
    return;
  }
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= a.x_chunks) return;                           // a multiple of 64: whole waves
  const int64_t piece = i >> 6, row = piece / a.r.nss;
  const int c = (int)(i & 63), col = (int)(piece - row * a.r.nss) * 512 + c * 8;
  uint32_t byte = 0;
  if (col < a.cols) {                                    // the same for a block's four lanes
    float x[8];
    load8<DT>(a.X, row * a.ldx + col, x);
    *(uint32_t*)(a.codes + row * (a.cols / 2) + col / 2) = quant8(x, byte);
  }
  const int blk = c >> 2;
  if ((c & 3) == 0) a.r.dst[0][piece * 16 + (blk & 3) * 4 + (blk >> 2)] = (uint8_t)byte;
}

// ---------------------------------------------------------------------------
// Many tokens: a workgroup of WM x WN waves owns tiles of TM tokens x TN weight
// rows, one after the other, and walks the contraction through LDS in stages of
// 256 elements (128 bytes of codes a row; with 64 bytes, half a line at a time,
// the loads cost 12% of the whole) of two product steps. A group of two stages
// shares the scales (reordered as above), which come with its first; NG groups
// are resident.
//
// Everything comes by 16-byte DMA. A lane's results are 8 consecutive outputs
// of a token: row i = 4 a + b of weight fragments 2 j and 2 j + 1 is LDS row
// 32 j + 8 a + b (+ 4), and chunk c (one block of 32) of an LDS row r sits at
// c ^ (r & 3 | (r & 8) / 2), X's at c ^ (r & 7), so that fragment reads use
// every bank equally. Rows past the end are out of the buffer's range and
// arrive as zeros; from stage to stage only the buffer's base and range move,
// not the lanes' offsets.
//
// During a step the next step's fragments are read. The barrier in the middle
// of a stage says that everyone has read all of it and that the next stage has
// landed; the DMAs of the stage 2 NG later then go where this one was, early in
// the step, and have most of two steps (of 1024 cycles at 256 x 256) to arrive.
// Loads run on into the next tile, and a tile's stores are waited for with the
// next tile's second stage.
//
// With one wave a SIMD (256 x 256) a product takes 16 cycles of the matrix core
// and 8 of the wave's issue, which leaves room for two other instructions: the
// scales by dword, the DMAs' constant offsets and the scalar base are for that.
// 4096 x 8192 x 28672 in 452 us, 4.25 PFLOP/s.
// ---------------------------------------------------------------------------

// One product step with its accumulator pinned to AGPRs (the compiler otherwise
// moves accumulators between the two halves of the register file all the
// time); J selects the scales' byte. The hazard recogniser does not look
// inside the asm: the sources are LDS loads, which the compiler waits for;
// code that reads the accumulators first waits out the instruction's latency
// (mfma_drain).
template <int J>
__device__ __forceinline__ void mfma_acc(f32x4& c, const i32x4& w, const i32x4& x, int ws, int xs) {
#define QAT_MX_MFMA(SEL)                                                              \
  asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 " SEL " cbsz:4 blgp:4" \
               : "+a"(c)                                                              \
               : "v"(w), "v"(x), "v"(ws), "v"(xs))
  if constexpr (J == 0) QAT_MX_MFMA("op_sel_hi:[0,0,0]");
  else if constexpr (J == 1) QAT_MX_MFMA("op_sel:[1,1,0] op_sel_hi:[0,0,0]");
  else if constexpr (J == 2) QAT_MX_MFMA("op_sel_hi:[1,1,0]");
  else QAT_MX_MFMA("op_sel:[1,1,0] op_sel_hi:[1,1,0]");
#undef QAT_MX_MFMA
}

// dma16 (qat_dma.h) to `lds` + `imm`, the sum formed in M0.
__device__ __forceinline__ void dma16_at(i32x4 rsrc, uint32_t lds, int imm, uint32_t voff) {
  asm volatile("s_add_u32 m0, %0, %1\n\tbuffer_load_dwordx4 %2, %3, 0 offen lds"
               :
               : "s"(lds), "n"(imm), "v"(voff), "s"(rsrc)
               : "memory", "m0", "scc");
}

__device__ __forceinline__ void mfma_drain() {
  asm volatile("s_nop 15\n\ts_nop 15\n\ts_nop 15" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

template <int TM, int TN, int WM, int WN, int NG>
struct TileShape {
  static constexpr int kWaves = WM * WN, kRows = TM + TN;
  static constexpr int kStage = kRows * 128;              // codes
  static constexpr int kGroup = 2 * kStage + kRows * 16;  // two stages, then their scales
  static constexpr int kLds = NG * kGroup;
  static constexpr int kDma = kRows / 8 / kWaves;         // DMAs of a wave: a stage's codes
  static constexpr int kSDma = (kRows / 64 + kWaves - 1) / kWaves;   // and a group's scales
  static_assert(kDma * kWaves * 8 == kRows && TM % 64 == 0 && TN % 64 == 0, "whole DMAs, one operand each");
  static_assert(kLds <= 160 * 1024, "LDS of a workgroup");
  static constexpr int kFlight = (NG - 1) * (2 * kDma + kSDma);      // DMAs behind the next stage at a barrier
  static constexpr int kStores = TM * TN / 8 / 64 / kWaves;          // of a wave's results
};

template <int DT, int TM, int TN, int WM, int WN, int NG>
__global__ __launch_bounds__(64 * WM * WN, 1) void k_mx_tile(const ProductArgs a) {
  typedef TileShape<TM, TN, WM, WN, NG> TS;
  constexpr int FM = TM / WM / 16, FN = TN / WN / 16;
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int wm = wave / WN, wn = wave - wm * WN;
  const int ldk = a.K / 2, SS = (a.K + 511) / 512;        // groups

  // Tiles of this workgroup: the grid has at most one workgroup for each CU and
  // walks the tiles in rounds. Consecutive tiles are on one XCD, in bands of up
  // to 4 token tiles, so that the tiles an XCD works on together share both
  // operands; the last round is what is left.
  const int tm = (a.M + TM - 1) / TM, tn = (a.N + TN - 1) / TN, T = tm * tn;
  const int xcd = blockIdx.x & 7, slot = blockIdx.x >> 3;
  const int xcd_tiles = (T >> 3) + (xcd < (T & 7) ? 1 : 0), xcd_first = xcd * (T >> 3) + min(xcd, T & 7);
  const int xcd_slots = ((int)gridDim.x + 7 - xcd) >> 3;
  auto tile_at = [&](int k, int& m0, int& n0) {           // tile k of this workgroup; false past its last
    const int local = k * xcd_slots + slot;
    if (local >= xcd_tiles) return false;
    constexpr int kBand = 4;
    const int id = xcd_first + local;
    const int band = id / (kBand * tn), in_band = id - band * kBand * tn;
    const int h = min(kBand, tm - band * kBand);
    m0 = (band * kBand + in_band % h) * TM;
    n0 = (in_band / h) * TN;
    return true;
  };
  i32x4 rx, rw, rxs, rws;
  auto open = [&](int k) {                                // the buffers at the start of tile k, or empty
    int m = 0, n = 0;
    const bool any = tile_at(k, m, n);
    const int rows_x = any ? min(TM, a.M - m) : 0, rows_w = any ? min(TN, a.N - n) : 0;
    rx = buffer_rsrc(a.xc + (int64_t)m * ldk, (int64_t)rows_x * ldk);
    rw = buffer_rsrc(a.wc + (int64_t)n * ldk, (int64_t)rows_w * ldk);
    rxs = buffer_rsrc(a.xs + (int64_t)m * SS * 16, (int64_t)rows_x * SS * 16);
    rws = buffer_rsrc(a.ws + (int64_t)n * SS * 16, (int64_t)rows_w * SS * 16);
  };
  // the next bytes of a buffer; empty once its end is passed
  auto advance = [](i32x4& r, uint32_t by) {
    const uint64_t b = ((uint64_t)(uint32_t)r[1] << 32 | (uint32_t)r[0]) + by;
    r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)b);
    r[1] = __builtin_amdgcn_readfirstlane((int)(b >> 32));
    r[2] = __builtin_amdgcn_readfirstlane(max(r[2] - (int)by, 0));
  };
  const uint32_t lds0 = lds_addr_of(smem);
  // DMA k of a stage moves rows 8 k .. + 7 (X's, then W's); lane l lands at row
  // l / 8, position l % 8, and fetches the chunk that this position holds
  uint32_t vc[TS::kDma], vs[TS::kSDma];
#pragma unroll
  for (int i = 0; i < TS::kDma; ++i) {
    const int k = wave * TS::kDma + i, r = lane >> 3;
    const bool is_x = k < TM / 8;
    const int row = (is_x ? k : k - TM / 8) * 8 + r, sw = is_x ? r : (r & 3) | (row & 8) >> 1;
    vc[i] = (uint32_t)(row * ldk + (((lane & 7) ^ sw) << 4));
    asm("" : "+v"(vc[i]));                                // kept, not formed again before each use
  }
#pragma unroll
  for (int i = 0; i < TS::kSDma; ++i) {
    const int k = wave * TS::kSDma + i;
    vs[i] = (uint32_t)(((k < TM / 64 ? k : k - TM / 64) * 64 + lane) * SS * 16);
  }
  // DMA i of the stage at which the buffers rx .. rws stand, into the LDS group
  // at `grp` as its stage j; from kDma on the group's scales
  auto issue = [&](uint32_t grp, int j, int i) {
    if (i < TS::kDma) {
      const int k = wave * TS::kDma + i;
      dma16_at(k < TM / 8 ? rx : rw, grp + (uint32_t)(wave * TS::kDma * 1024), j * TS::kStage + i * 1024, vc[i]);
    } else {
      // a wave without a share repeats the last one, so that all waves count alike
      const int k = min(wave * TS::kSDma + i - TS::kDma, TS::kRows / 64 - 1);
      const uint32_t v = (TS::kRows / 64) % TS::kWaves == 0 ? vs[i - TS::kDma]
                                                            : (uint32_t)(((k < TM / 64 ? k : k - TM / 64) * 64 + lane) * SS * 16);
      dma16(k < TM / 64 ? rxs : rws,
            (uint32_t)__builtin_amdgcn_readfirstlane((int)(grp + (uint32_t)(2 * TS::kStage + k * 1024))), v);
    }
  };
  auto next_stage = [&](bool group) {
    advance(rx, 128);
    advance(rw, 128);
    if (group) {
      advance(rxs, 16);
      advance(rws, 16);
    }
  };

  // step parity h of a stage: lane group g has chunk 4 h + g; weight fragments
  // 2 j + b are 32 j + 4 b rows in, with rows 8 (r16 / 4) + r16 % 4
  const int wrow = 8 * (r16 >> 2) + (r16 & 3), wsw = (r16 & 3) | (r16 & 4);
  const int xpos[2] = {(g ^ (r16 & 7)) << 4, ((4 + g) ^ (r16 & 7)) << 4};
  const int wpos[2] = {(g ^ wsw) << 4, ((4 + g) ^ wsw) << 4};
  const uint8_t* fx = smem + (wm * FM * 16 + r16) * 128;
  const uint8_t* fw = smem + (TM + wn * FN * 16 + wrow) * 128;
  const uint8_t* sx = smem + 2 * TS::kStage + (wm * FM * 16 + r16) * 16 + 4 * g;
  const uint8_t* sw = smem + 2 * TS::kStage + (TM + wn * FN * 16 + wrow) * 16 + 4 * g;

  struct Frags {
    i32x4 x[FM], w[FN];
  };
  struct Scales {
    int x[FM], w[FN];
  };
  // read r of a step, in the order in which the products use them: w0, x0 .. x(FM-1), w1 ..
  auto read = [&](Frags& f, int off, int h, int r) {
    if (r >= 1 && r <= FM) {
      f.x[r - 1] = *(const i32x4*)(fx + off + xpos[h] + (r - 1) * 2048);
    } else {
      const int i = r ? r - FM : 0;
      f.w[i] = *(const i32x4*)(fw + off + wpos[h] + (32 * (i >> 1) + 4 * (i & 1)) * 128);
    }
  };
  auto read_scale = [&](Scales& f, int off, int r) {
    if (r >= 1 && r <= FM) {
      f.x[r - 1] = *(const int*)(sx + off + (r - 1) * 256);
    } else {
      const int i = r ? r - FM : 0;
      f.w[i] = *(const int*)(sw + off + (32 * (i >> 1) + 4 * (i & 1)) * 16);
    }
  };
  f32x4 acc[FN][FM];
  constexpr int NM = FM * FN, NR = FM + FN;
  static_assert(NR <= NM, "a step's reads fit its products");
  // Step J of a group (scale byte J): product t, then read t of the next step
  // (from LDS offset `off`; its scales too where a group begins) and a share of
  // the DMAs (odd steps, into stage J / 2 of the group at `grp`). The DMAs of a
  // CU's four waves pass its L1 at 64 bytes a cycle, a stage in 1088 of its 2048
  // cycles: all at the step's start they stall their waves, so they are spread.
  // The fences keep this order: without them the compiler puts every read right
  // before its use.
  auto step = [&](auto jc, const Frags& cur, const Scales& sc, Frags& nxt, int off, Scales& nsc, int soff,
                  uint32_t grp) {
    constexpr int J = decltype(jc)::value;
    constexpr int ND = J % 2 == 0 ? 0 : TS::kDma + (J == 1 ? TS::kSDma : 0);
    constexpr int kGap = ND > 0 && NM / ND > 1 ? NM / ND : 1;         // products from one DMA to the next
    constexpr int kDmas = (ND + NM - 1) / NM;                         // and DMAs at a time, where there are more
    // a read with every product (more where there are too few products for one each)
    constexpr int kReads = (NR + NM - 1) / NM;
#pragma unroll
    for (int t = 0; t < NM; ++t) {
      const int j = t / FM, i = t % FM;
      mfma_acc<J>(acc[j][i], cur.w[j], cur.x[i], sc.w[j], sc.x[i]);
      if (t % kGap == 0) {
#pragma unroll
        for (int d = t / kGap * kDmas; d < (t / kGap + 1) * kDmas && d < ND; ++d) issue(grp, J / 2, d);
      }
#pragma unroll
      for (int r = t * kReads; r < (t + 1) * kReads && r < NR; ++r) {
        read(nxt, off, (J + 1) % 2, r);
        if constexpr (J == 3) read_scale(nsc, soff, r);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (J % 2) next_stage(J == 1);
  };
  // the barrier in a stage's middle; `stores`: a tile's stores are behind the next stage's DMAs
  auto landed = [&](bool stores) {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");    // this wave has read all of the stage
    constexpr int kMost = TS::kFlight + TS::kStores < 63 ? TS::kFlight + TS::kStores : 63;
    if (stores) wait_vmcnt<kMost>();
    else wait_vmcnt<TS::kFlight>();                       // its part of the next one has landed
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  constexpr std::integral_constant<int, 0> c0;
  constexpr std::integral_constant<int, 1> c1;
  constexpr std::integral_constant<int, 2> c2;
  constexpr std::integral_constant<int, 3> c3;

  // The loads run on from one tile into the next (and past the last tile from
  // empty buffers, as zeros): the next tile's first groups arrive while this
  // one's last are multiplied and its results are stored.
  int ahead = 0, ahead_ss = 0;                            // tile and group at which the buffers stand
  auto next_group = [&]() {
    if (++ahead_ss == SS) {
      asm volatile("");                                   // a branch: not computed and selected every time
      ahead_ss = 0;
      open(++ahead);
    }
  };
  open(0);
#pragma unroll
  for (int i = 0; i < 2 * NG; ++i) {
#pragma unroll
    for (int d = 0; d < TS::kDma + (i % 2 ? 0 : TS::kSDma); ++d) issue(lds0 + (uint32_t)(i / 2 * TS::kGroup), i % 2, d);
    next_stage(i % 2 == 0);
    if (i % 2) next_group();
  }
  wait_vmcnt<TS::kFlight + TS::kDma>();                   // stage 0
  __syncthreads();
  Frags p, q;
  Scales sc, nsc;
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    read(p, 0, 0, r);
    read_scale(sc, 0, r);
  }
  __builtin_amdgcn_sched_barrier(0);
  int off = 0;                                            // LDS offset of the group
  bool stores = false;                                    // the last tile's, all of kStores or more, may be on their way
  int m0, n0;
  for (int k = 0; tile_at(k, m0, n0); ++k) {
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int i = 0; i < FM; ++i) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    mfma_drain();                                         // written before the first product reads them
#pragma clang loop unroll(disable)
    for (int ss = 0; ss < SS; ++ss) {
      const int nxt = NG == 1 || off == (NG - 1) * TS::kGroup ? 0 : off + TS::kGroup;
      const uint32_t grp = lds0 + (uint32_t)off;
      step(c0, p, sc, q, off, nsc, 0, grp);
      landed(stores && ss == 0);
      step(c1, q, sc, p, off + TS::kStage, nsc, 0, grp);
      step(c2, p, sc, q, off + TS::kStage, nsc, 0, grp);
      landed(false);
      step(c3, q, sc, p, nxt, nsc, nxt, grp);
      next_group();
      sc = nsc;
      off = nxt;
      // nothing behind the loop may read a result before it is written
      if (ss == SS - 1) mfma_drain();
    }
    mfma_drain();
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int m = m0 + (wm * FM + i) * 16 + r16;
      if (m < a.M) {
#pragma unroll
        for (int j = 0; j < FN; j += 2)
          store_out8<DT>(a.Y, a.ldy, m, n0 + (wn * FN + j) * 16 + 8 * g, a.N, acc[j][i], acc[j + 1][i]);
      }
    }
    // a tile over the edge may have stored less: then the count would not hold
    stores = m0 + TM <= a.M && n0 + TN <= a.N;
  }
  wait_vmcnt<0>();                                        // the DMAs past the last tile
}

// ---------------------------------------------------------------------------
// Launchers
// ---------------------------------------------------------------------------
void launch_quant(const void* X, int dtype, int64_t rows, int64_t cols, int64_t ldx, uint8_t* codes, uint8_t* scales,
                  void* x_hat, hipStream_t st) {
  QuantArgs a;
  a.X = X;
  a.ldx = ldx;
  a.chunks = (uint32_t)(rows * (cols / 8));
  a.row_chunks = (uint32_t)(cols / 8);
  a.div = FastDiv::make(a.row_chunks);
  a.codes = codes;
  a.scales = scales;
  a.x_hat = x_hat;
  LaunchTimer t("mx_quant", st);
  const dim3 grid((a.chunks + 255) / 256);
  if (dtype == QAT_F32) QAT_LAUNCH(k_mx_quant<QAT_F32>, grid, dim3(256), 0, st, a);
  else if (dtype == QAT_BF16) QAT_LAUNCH(k_mx_quant<QAT_BF16>, grid, dim3(256), 0, st, a);
  else QAT_LAUNCH(k_mx_quant<QAT_F16>, grid, dim3(256), 0, st, a);
}

// Compute units of the current device.
int num_cus() {
  static int cached[64] = {0};
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
  if (!cached[dev]) {
    int n = 0;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0) n = 256;
    cached[dev] = n;
  }
  return cached[dev];
}

// Whether a product takes the tiled kernel. The other one reads its operands in
// place, which spares the scales' reordering, but reads the weights again for
// every 16 tokens: measured at 2.7 us for each 2^20 of (token tiles x weight
// tiles x in), against 14 to 15 us in all for the smallest tiled products of
// 4096 and more (32 x 4096 x 4096: 6 us against 14; 32 x 11008 x 4096: 15
// against 15; 128 x 4096 x 4096: 20 against 14).
bool tiled(int64_t M, int64_t out, int64_t in) {
  if ((M + 15) / 16 > 65535) return true;                 // the other one's grid
  return M > 16 && (M + 15) / 16 * ((out + 15) / 16) * in > (int64_t(11) << 19);
}

template <int DT, int TM, int TN, int WM, int WN, int NG>
void launch_tile(const ProductArgs& a, hipStream_t st) {
  typedef TileShape<TM, TN, WM, WN, NG> TS;
  (void)hipFuncSetAttribute((const void*)k_mx_tile<DT, TM, TN, WM, WN, NG>,
                            hipFuncAttributeMaxDynamicSharedMemorySize, TS::kLds);
  const int64_t tiles = (int64_t)((a.M + TM - 1) / TM) * ((a.N + TN - 1) / TN);
  const int64_t slots = (int64_t)num_cus() * (160 * 1024 / TS::kLds);
  QAT_LAUNCH((k_mx_tile<DT, TM, TN, WM, WN, NG>), dim3((unsigned)(tiles < slots ? tiles : slots)),
             dim3(64 * TS::kWaves), TS::kLds, st, a);
}

// Tile by how many there are for the chip (measured on 256 CUs, us, 64 x 64 /
// 128 x 128 one group / two groups / 256 x 256):
//   256 x 4096 x 4096       64 tiles of 128^2   11 / 16 / 15 / 29
//   1024 x 4096 x 4096     256                  23 / 18 / 17 / 30
//   2048 x 4096 x 11008    512                  97 / 55 / 57 / 67
//   4096 x 8192 x 8192    2048                 283 / 148 / 165 / 123
template <int DT>
void launch_tiles(const ProductArgs& a, hipStream_t st) {
  auto tiles = [&](int64_t t) { return (a.M + t - 1) / t * ((a.N + t - 1) / t); };
  const int cus = num_cus();
  if (tiles(256) >= cus) launch_tile<DT, 256, 256, 2, 2, 1>(a, st);
  else if (tiles(128) > cus) launch_tile<DT, 128, 128, 2, 2, 1>(a, st);        // two workgroups a CU
  else if (2 * tiles(128) > cus) launch_tile<DT, 128, 128, 2, 2, 2>(a, st);    // one: twice the depth
  else launch_tile<DT, 64, 64, 2, 2, 2>(a, st);
}

// Workspace: X's codes (qat_mx_linear), then both operands' scales in the tiled
// kernel's order, or X's as they are for the other one.
struct MxWs {
  size_t xs, ws, bytes;
  static MxWs of(int64_t M, int64_t out, int64_t in, bool linear) {
    auto up = [](int64_t v) { return (size_t)((v + 255) / 256 * 256); };
    const int64_t row = (in + 511) / 512 * 16;
    const bool tile = tiled(M, out, in);
    if (M <= kQuantTokens) linear = false;                // X is quantised in the product
    MxWs w;
    w.xs = linear ? up(M * in / 2) : 0;
    w.ws = w.xs + (tile ? up(M * row) : linear ? up(M * in / 32) : 0);
    w.bytes = w.ws + (tile ? up(out * row) : 0);
    return w;
  }
};

ReorderArgs reorder_args(const ProductArgs& a, uint8_t* ws, const MxWs& w) {
  ReorderArgs r;
  r.nblk = a.K / 32;
  r.nss = (r.nblk + 15) / 16;
  r.src[0] = a.xs;
  r.src[1] = a.ws;
  r.dst[0] = ws + w.xs;
  r.dst[1] = ws + w.ws;
  r.n0 = (int64_t)a.M * r.nss;
  r.n1 = (int64_t)a.N * r.nss;
  return r;
}

// The product proper: `a` has tiled scales where tiled() says so.
void launch_product(const ProductArgs& a, int dtype, hipStream_t st) {
  LaunchTimer t("mx_gemm", st);
  if (tiled(a.M, a.N, a.K)) {
    if (dtype == QAT_BF16) launch_tiles<QAT_BF16>(a, st);
    else launch_tiles<QAT_F16>(a, st);
    return;
  }
  const dim3 grid((a.N + 15) / 16, (a.M + 15) / 16);
  if (a.x16) {
    if (dtype == QAT_BF16) QAT_LAUNCH((k_mx_skinny<QAT_BF16, true>), grid, dim3(512), 0, st, a);
    else QAT_LAUNCH((k_mx_skinny<QAT_F16, true>), grid, dim3(512), 0, st, a);
  } else {
    if (dtype == QAT_BF16) QAT_LAUNCH((k_mx_skinny<QAT_BF16, false>), grid, dim3(512), 0, st, a);
    else QAT_LAUNCH((k_mx_skinny<QAT_F16, false>), grid, dim3(512), 0, st, a);
  }
}

void launch_gemm(ProductArgs a, int dtype, uint8_t* ws, const MxWs& w, hipStream_t st) {
  if (tiled(a.M, a.N, a.K)) {
    const ReorderArgs r = reorder_args(a, ws, w);
    {
      LaunchTimer t("mx_reorder", st);
      QAT_LAUNCH(k_mx_reorder, dim3((unsigned)((r.n0 + r.n1 + 255) / 256)), dim3(256), 0, st, r);
    }
    a.xs = r.dst[0];
    a.ws = r.dst[1];
  }
  launch_product(a, dtype, st);
}

void launch_linear(const void* X, int64_t ldx, ProductArgs a, int dtype, uint8_t* ws, const MxWs& w, hipStream_t st) {
  if (a.M <= kQuantTokens) {
    a.x16 = X;
    a.ldx = ldx;
    launch_product(a, dtype, st);
    return;
  }
  a.xc = ws;
  a.xs = ws + w.xs;
  if (tiled(a.M, a.N, a.K)) {
    PrepareArgs p;
    p.X = X;
    p.ldx = ldx;
    p.cols = a.K;
    p.codes = ws;
    p.r = reorder_args(a, ws, w);
    p.x_chunks = p.r.n0 * 64;
    p.x_blocks = (int)((p.x_chunks + 255) / 256);
    {
      LaunchTimer t("mx_prepare", st);
      const dim3 grid((unsigned)(p.x_blocks + (p.r.n1 + 255) / 256));
      if (dtype == QAT_BF16) QAT_LAUNCH(k_mx_prepare<QAT_BF16>, grid, dim3(256), 0, st, p);
      else QAT_LAUNCH(k_mx_prepare<QAT_F16>, grid, dim3(256), 0, st, p);
    }
    a.ws = p.r.dst[1];
  } else {
    launch_quant(X, dtype, a.M, a.K, ldx, ws, ws + w.xs, nullptr, st);
  }
  launch_product(a, dtype, st);
}

int32_t check_product(int64_t M, int64_t out, int64_t in, int32_t dtype, int64_t ldy) {
  if (dtype != QAT_BF16 && dtype != QAT_F16) return QAT_ERR_TYPE;
  if (M < 0 || out <= 0 || in <= 0 || in % 32 != 0) return QAT_ERR_SHAPE;
  if (M > kMaxCount || out > kMaxCount || in > (1 << 20) || ldy < out || ldy > kMaxCount) return QAT_ERR_SHAPE;
  if (M * in * 2 > kMaxOperandBytes || out * in / 2 > kMaxOperandBytes || M * ldy * 2 > kMaxOperandBytes)
    return QAT_ERR_SHAPE;
  return QAT_OK;
}

}  // namespace
}  // namespace qat

QAT_API int32_t qat_mx_quant(const void* X, int32_t dtype, int64_t rows, int64_t cols, int64_t ldx, uint8_t* codes,
                             uint8_t* scales, void* X_hat, hipStream_t stream) {
  using namespace qat;
  if (dtype < QAT_F32 || dtype > QAT_F16) return QAT_ERR_TYPE;
  const int64_t e = dtype == QAT_F32 ? 4 : 2;
  if (rows < 0 || cols <= 0 || cols % 32 != 0 || rows > kMaxCount || cols > kMaxCount || ldx < cols ||
      ldx > kMaxCount || rows * (cols / 8) >= (int64_t(1) << 31))
    return QAT_ERR_SHAPE;
  if (rows == 0) return QAT_OK;
  if (!X || (!codes && !X_hat) || !codes != !scales) return QAT_ERR_NULL;
  if ((ldx * e) % 16 != 0) return QAT_ERR_ALIGN;
  QAT_CHECK(check_aligned({X, codes, scales, X_hat}));
  QAT_CHECK(check_spans({{codes, (size_t)(rows * cols / 2)}, {scales, (size_t)(rows * cols / 32)},
                         {X_hat, (size_t)(rows * cols * e)}},
                        {{X, strided_bytes(rows, ldx, cols, e)}}));
  launch_quant(X, dtype, rows, cols, ldx, codes, scales, X_hat, stream);
  return finish_call();
}

QAT_API size_t qat_mx_ws_bytes(int64_t M, int64_t out, int64_t in) {
  using namespace qat;
  if (check_product(M, out, in, QAT_BF16, out) != QAT_OK) return 0;
  return MxWs::of(M, out, in, true).bytes;
}

QAT_API int32_t qat_mx_gemm(const uint8_t* X_codes, const uint8_t* X_scales, const uint8_t* W_codes,
                            const uint8_t* W_scales, int64_t M, int64_t out, int64_t in, int32_t dtype, void* Y,
                            int64_t ldy, void* ws, size_t ws_bytes, hipStream_t stream) {
  using namespace qat;
  QAT_CHECK(check_product(M, out, in, dtype, ldy));
  if (M == 0) return QAT_OK;
  const MxWs w = MxWs::of(M, out, in, false);
  if (w.bytes && (!ws || ws_bytes < w.bytes)) return QAT_ERR_WORKSPACE;
  QAT_CHECK(check_required({X_codes, X_scales, W_codes, W_scales, Y}));
  QAT_CHECK(check_aligned({X_codes, X_scales, W_codes, W_scales, Y, ws}));
  QAT_CHECK(check_spans({{Y, strided_bytes(M, ldy, out, 2)}, {ws, w.bytes}},
                        {{X_codes, (size_t)(M * in / 2)}, {X_scales, (size_t)(M * in / 32)},
                         {W_codes, (size_t)(out * in / 2)}, {W_scales, (size_t)(out * in / 32)}}));
  ProductArgs a{X_codes, X_scales, W_codes, W_scales, (int)M, (int)out, (int)in, Y, ldy, nullptr, 0};
  launch_gemm(a, dtype, (uint8_t*)ws, w, stream);
  return finish_call();
}

QAT_API int32_t qat_mx_linear(const void* X, int64_t ldx, const uint8_t* W_codes, const uint8_t* W_scales, int64_t M,
                              int64_t out, int64_t in, int32_t dtype, void* Y, int64_t ldy, void* ws,
                              size_t ws_bytes, hipStream_t stream) {
  using namespace qat;
  QAT_CHECK(check_product(M, out, in, dtype, ldy));
  if (ldx < in || ldx > kMaxCount || M * ldx * 2 > kMaxOperandBytes) return QAT_ERR_SHAPE;
  if (M == 0) return QAT_OK;
  QAT_CHECK(check_required({X, W_codes, W_scales, Y}));
  if (ldx % 8 != 0) return QAT_ERR_ALIGN;
  QAT_CHECK(check_aligned({X, W_codes, W_scales, Y, ws}));
  const MxWs w = MxWs::of(M, out, in, true);
  if (w.bytes && (!ws || ws_bytes < w.bytes)) return QAT_ERR_WORKSPACE;
  QAT_CHECK(check_spans({{Y, strided_bytes(M, ldy, out, 2)}, {ws, w.bytes}},
                        {{X, strided_bytes(M, ldx, in, 2)}, {W_codes, (size_t)(out * in / 2)},
                         {W_scales, (size_t)(out * in / 32)}}));
  ProductArgs a{nullptr, nullptr, W_codes, W_scales, (int)M, (int)out, (int)in, Y, ldy, nullptr, 0};
  launch_linear(X, ldx, a, dtype, (uint8_t*)ws, w, stream);
  return finish_call();
}
