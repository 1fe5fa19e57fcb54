// MXFP4 path for gfx950: quantize (bf16 -> E2M1 codes with one E8M0 scale per 32 elements),
// dequantize, and the product of two MXFP4 operands on the block-scaled MFMA.
//
// MXFP4 is the 4-bit member of the Open Compute Project's microscaling formats: E2M1
// elements in 32-element blocks that share one power-of-two scale. A block's shared
// exponent is e = floor(log2(amax)) - 2 (2 = the exponent of the largest E2M1 value,
// 6 = 1.5 * 2^2) clamped to [-127, 127], stored as the byte e + 127; an all-zero block
// takes byte 0, and a block that holds a NaN or an infinity takes byte 0xFF, the scale
// format's NaN, so that it reads back as NaN. Elements are the E2M1 value nearest to
// x / 2^e, ties to the even code, saturating at 6, sign copied.
#include <type_traits>

#include "gemm_common.hpp"
#include "mx4_offsets.hpp"

namespace nvfp4 {

namespace {

typedef int v8i_t __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));

// Scale byte of a block from the largest bf16 magnitude pattern in it (sign bits cleared):
// the exponent field less 2, zero for zero and subnormal maxima (whose floor(log2) is at
// most -127), 0xFF for infinities and NaN.
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t amax16) {
  const int field = (int)(amax16 >> 7);
  return field == 0xFF ? 0xFFu : (uint32_t)max(field - 2, 0);
}

// The scale of byte b as the binary32 operand of gfx950's scaled conversions, which take
// its exponent field alone: field 0 stands for 2^-127 and field 255 for NaN.
__device__ __forceinline__ float mx4_scale_operand(uint32_t b) { return u2f(b << 23); }

// ---- quantize ----------------------------------------------------------------------
//
// Four lanes share a block: lane 4i+q holds elements [8q, 8q+8) of block i. The block's
// maximum is taken on the bf16 bit patterns (for magnitudes their integer order is the order
// of the values), and each lane converts its elements with the scaled conversion from bf16
// (x / 2^e, nearest even, saturating: equal to the rule above for every bf16 value and
// scale) into 4 bytes of codes.
struct Mx4Codes {
  uint32_t word, byte;
};
__device__ __forceinline__ Mx4Codes mx4_encode_quad(const u32x4 v) {
  uint32_t a = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a = max(a, v[i] & 0x7FFFu);
    a = max(a, (v[i] >> 16) & 0x7FFFu);
  }
  // quad maximum: DPP quad_perm [1,0,3,2], then [2,3,0,1]
  a = max(a, (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0xB1, 0xF, 0xF, false));
  a = max(a, (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0x4E, 0xF, 0xF, false));
  const uint32_t byte = mx4_scale_byte(a);
  const float s = mx4_scale_operand(byte);
  // each pair through an integer of its own: __builtin_bit_cast of a vector's element takes
  // the first element whatever the index (this toolchain)
  const uint32_t x0 = v.x, x1 = v.y, x2 = v.z, x3 = v.w;
  uint32_t w = 0u;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2_t, x0), s, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2_t, x1), s, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2_t, x2), s, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2_t, x3), s, 3);
  return Mx4Codes{byte == 0xFFu ? 0u : w, byte};  // a NaN block's codes are 0
}

// Memory-bound: 2 B read, 1/2 + 1/32 B written per element; a lane loads 16 bytes, so that a
// wave's load reads 1 KiB of consecutive bytes.
template <int UNROLL>
__global__ void __launch_bounds__(256) mx4_quantize_kernel(const u32x4* __restrict__ x,
                                                           uint32_t* __restrict__ packed,
                                                           uint8_t* __restrict__ scales,
                                                           int64_t nlanes) {
  const int64_t stride = (int64_t)gridDim.x * blockDim.x * UNROLL;
  for (int64_t base = (int64_t)blockIdx.x * blockDim.x * UNROLL + threadIdx.x; base < nlanes;
       base += stride) {
    u32x4 v[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int64_t li = base + (int64_t)u * blockDim.x;
      v[u] = li < nlanes ? __builtin_nontemporal_load(&x[li]) : u32x4{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      // nlanes is a multiple of 4: the lanes of a quad are in or out of range together
      const int64_t li = base + (int64_t)u * blockDim.x;
      const Mx4Codes c = mx4_encode_quad(v[u]);
      if (li < nlanes) {
        __builtin_nontemporal_store(c.word, &packed[li]);
        if ((li & 3) == 0) scales[li >> 2] = (uint8_t)c.byte;
      }
    }
  }
}

// ---- dequantize ----------------------------------------------------------------------
//
// Memory-bound the other way: a lane reads 8 codes (4 bytes) and its block's scale byte
// and stores 8 bf16 values (16 bytes). E2M1 times a power of two is exact in bf16 (also
// among its subnormals); only 2^126 and 2^127 times 4 and 6 exceed its range, and become
// infinities.
template <int UNROLL>
__global__ void __launch_bounds__(256) mx4_dequantize_kernel(const uint32_t* __restrict__ packed,
                                                             const uint8_t* __restrict__ scales,
                                                             u32x4* __restrict__ out,
                                                             int64_t nlanes) {
  const int64_t stride = (int64_t)gridDim.x * blockDim.x * UNROLL;
  for (int64_t base = (int64_t)blockIdx.x * blockDim.x * UNROLL + threadIdx.x; base < nlanes;
       base += stride) {
    uint32_t c[UNROLL], b[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int64_t li = base + (int64_t)u * blockDim.x;
      c[u] = li < nlanes ? packed[li] : 0u;
      b[u] = li < nlanes ? scales[li >> 2] : 0u;
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int64_t li = base + (int64_t)u * blockDim.x;
      const float s = mx4_scale_operand(b[u]);
      u32x4 o;
      o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[u], s, 0));
      o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[u], s, 1));
      o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[u], s, 2));
      o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[u], s, 3));
      if (li < nlanes) __builtin_nontemporal_store(o, &out[li]);
    }
  }
}

// ---- GEMM ----------------------------------------------------------------------------
//
// out[M, N] (bf16) = A_hat[M, K] W_hat[N, K]^T. v_mfma_scale_f32_32x32x64_f8f6f4 takes
// E2M1 operands and E8M0 scales as stored: over a 64-element step, lane (h, r) =
// (lane / 32, lane % 32) of an operand holds the 32 elements of row r's block h (16
// bytes) and that block's scale byte. The weights are its A operand, so that a lane's
// results are four neighbouring columns of one output row.
// ---- GEMM, tiles through LDS ----------------------------------------------------------
//
// BM x BN output tiles, four waves of (BM / WM) x (BN / WN) each in blocks of 32 x 32. K
// goes by stages of 256 elements: a 128-byte line of codes per row, loaded direct to LDS
// eight rows at a time (8 lanes per row; such loads cost by the lines they touch), and 8
// scale bytes. A lane (h, r) of step s = 0..3 of a stage takes block 4h + s: 16 bytes of
// codes at chunk 4h + s of its row, and byte s of the row's scale word h, which the MFMA
// selects itself, so a lane reads one scale word per row and stage. (Any order of K serves
// as long as both operands share it.)
//
// LDS rows of 128 bytes hold chunk c at slot c ^ x_swz(row % 32), which keeps the fragment
// reads of a half wave in distinct banks. NBUF stage buffers; scales sit in two buffers of
// two stages (16 bytes per row) each, which a thread per row fills through registers: K / 32
// bytes of a row may start at any byte, and a register load has no alignment to keep.
//
// Pipeline. During step s a wave multiplies the fragments of step s and reads those of step
// s + 1. In step 3 of stage t, after its first MFMAs, it waits until the loads of stage t + 1
// have landed and meets the workgroup at a barrier: from there on stage t + 1 is readable by
// all, and buffer t % NBUF, whose last fragments everyone holds in registers, takes the loads
// of stage t + NBUF under the other MFMAs.
//
// Ragged ends: rows past M or N, and chunks of 32 elements past K, read as zero (their
// per-lane offset lies past the operand's window); scales past K are not loaded.
//
// KS > 1: KS groups of four waves each take a part of K, with buffers of their own, and add up
// in LDS at the end: for products of fewer tiles than compute units. Every part but the last
// has to have two stages (16 scale bytes) of its own, or its scale reads would start before
// the row: KS = 2 takes K > 1024.
template <int BM, int BN, int NBUF>
struct alignas(16) Mx4Smem {
  uint8_t x[NBUF][BM * 128];
  uint8_t w[NBUF][BN * 128];
  uint8_t sc[2][(BM + BN) * 16];
};

// Workgroup -> tile: as tile_order, for any number of tiles (an XCD's share of the order is
// contiguous whatever the remainder).
__device__ __forceinline__ void mx4_tile_order(int b, int tiles_m, int tiles_n, int& tm, int& tn) {
  constexpr int kXcd = 8, G = NVFP4_GEMM_XCD_GROUP;
  const int T = tiles_m * tiles_n, x = b % kXcd;
  const int q = x * (T / kXcd) + min(x, T % kXcd) + b / kXcd;
  const int per_group = G * tiles_n;
  const int gm0 = (q / per_group) * G;
  const int rows = min(tiles_m - gm0, G);
  const int r = q % per_group;
  tm = gm0 + r % rows;
  tn = r / rows;
}

// Scale bytes of a row's cut end: v holds the row's last 16 bytes, of which the first `cut`
// belong to the quarter before; shifted down, zeros behind.
__device__ __forceinline__ u32x4 mx4_cut_scales(const u32x4 v, uint32_t cut) {
  uint32_t w[5] = {v.x, v.y, v.z, v.w, 0u};
  if (cut & 8u) w[0] = w[2], w[1] = w[3], w[2] = w[3] = 0u;
  if (cut & 4u) w[0] = w[1], w[1] = w[2], w[2] = w[3], w[3] = 0u;
  return u32x4{__builtin_amdgcn_alignbyte(w[1], w[0], cut & 3u), __builtin_amdgcn_alignbyte(w[2], w[1], cut & 3u),
               __builtin_amdgcn_alignbyte(w[3], w[2], cut & 3u), __builtin_amdgcn_alignbyte(w[4], w[3], cut & 3u)};
}

// Stores of a wave's blocks: as store_tile_lds (rounded through the wave's own LDS area, 16
// bytes of a row per lane), with 16-byte stores at any alignment, since N need not be even.
template <int FM, int FN>
__device__ __forceinline__ void mx4_store_tile(const floatx16 (&acc)[FN][FM], const GemmProblem& p,
                                               int64_t m_base, int64_t n_base, int lane, uint16_t* area) {
  constexpr int W = FN * 32, RS = kStoreRowPad(FN);
  constexpr int kPieces = 32 * W / 8;
  const int h = lane >> 5, r32 = lane & 31;
  const bool aligned16 = (p.N & 7) == 0;
#pragma unroll
  for (int g = 0; g < FM; ++g) {
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *(u32x2*)&area[r32 * RS + i * 32 + 8 * q + 4 * h] =
            bf16x4_rne(acc[i][g][4 * q], acc[i][g][4 * q + 1], acc[i][g][4 * q + 2], acc[i][g][4 * q + 3]);
    static_assert(kPieces % 64 == 0, "whole turns");
#pragma unroll
    for (int it = 0; it < kPieces / 64; ++it) {
      const int c = it * 64 + lane;
      const int r = c / (W / 8), col = (c % (W / 8)) * 8;
      const int64_t m = m_base + g * 32 + r, n = n_base + col;
      if (m < p.M && n < p.N) {
        const u32x4 v = *(const u32x4*)&area[r * RS + col];
        uint16_t* o = p.out + m * p.N + n;
        if (n + 7 < p.N) {
          if (aligned16) __builtin_nontemporal_store(v, (u32x4*)o);
          else __builtin_memcpy(o, &v, 16);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (n + e < p.N) o[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
        }
      }
    }
  }
}

template <int BM, int BN, int NBUF, int KS>
__global__ void __launch_bounds__(256 * KS) gemm_mx4_kernel(GemmProblem p) {
  constexpr int NW = 4, WM = 2, WN = 2;
  __shared__ Mx4Smem<BM, BN, NBUF> smem[KS];
  constexpr int WTM = BM / WM, WTN = BN / WN;
  constexpr int FM = WTM / 32, FN = WTN / 32;
  constexpr int kPx = BM / 8 / NW, kPw = BN / 8 / NW;  // 1 KiB pieces per wave and stage
  constexpr int kLoads = kPx + kPw;
  constexpr int kRows = (BM + BN) / 64;                // scale rows that a lane loads of
  // loads of a stage issued by the end of steps 3, 0, 1 and 2
  constexpr int kL3 = kLoads * 3 / 8, kL0 = kLoads * 6 / 8, kL1 = kLoads * 8 / 8;
  constexpr int kMfma = FN * FM;
  constexpr int kFrags = FN + FM;
  constexpr int kHalf = kMfma >= 16 ? 4 : kMfma > 1 ? 1 : 0;  // MFMAs of step 3 before its barrier
  constexpr int kWait = (NBUF - 2) * kLoads;           // loads that may be in flight there

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((threadIdx.x >> 6) & 3);
  const int part = KS == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
  Mx4Smem<BM, BN, NBUF>& sm = smem[part];
  const int wave_n = wave % WN, wave_m = wave / WN;
  const int h = lane >> 5, r32 = lane & 31;

  int tile_m, tile_n;
  mx4_tile_order(blockIdx.x, (int)((p.M + BM - 1) / BM), (int)((p.N + BN - 1) / BN), tile_m, tile_n);
  const int64_t m0 = (int64_t)tile_m * BM, n0 = (int64_t)tile_n * BN;
  const int knb = (int)(p.K >> 5);           // blocks (16-byte chunks, scale bytes) per row
  const Mx4Part kp = mx4_part(knb, KS, part);
  const int nst = kp.nst, s0 = kp.s0, nb = kp.nb;
  const uint32_t pitch = (uint32_t)p.K >> 1;

  // windows of the tile's rows, at most BM (BN) of them: 32-bit offsets for any M, N
  const __amdgpu_buffer_rsrc_t rx = window_rsrc(p.a_packed, m0, min(p.M, m0 + BM), pitch);
  const __amdgpu_buffer_rsrc_t rw = window_rsrc(p.w_packed, n0, min(p.N, n0 + BN), pitch);
  // piece i = j * NW + wave covers rows 8i .. 8i + 7; its chunk order depends on i's parity
  // alone (NW is even), so on the wave
  const int lrow = 8 * wave + (lane >> 3);
  const int chunk = mx4_chunk(lane, lrow);
  const uint32_t voff = mx4_code_voff(lrow, chunk, pitch);
  auto issue_code = [&](int j, int stage, int buf) {
    const uint32_t v = voff | mx4_code_mask(stage, chunk, nb);
    if (j < kPx)
      buffer_load_lds16(rx, &sm.x[buf][(j * NW + wave) * 1024], v + (uint32_t)(j * NW * 8) * pitch, (uint32_t)(s0 + stage) * 128);
    else
      buffer_load_lds16(rw, &sm.w[buf][((j - kPx) * NW + wave) * 1024], v + (uint32_t)((j - kPx) * NW * 8) * pitch, (uint32_t)(s0 + stage) * 128);
  };

  // Scale rows: activation rows first, then weight rows; four lanes load 64 bytes of a row
  // (8 stages) and hold them in registers, and one of them at a time, a quarter, stores its 16
  // bytes (2 stages) for the multiplications. Rows past the end take the last row's (their
  // codes are zero).
  u32x4 sreg[kRows];
  const int quarter = lane & 3;
  const int srow = 16 * wave + (lane >> 2);
  const uint8_t* xsb = p.a_scales + m0 * knb;
  const uint8_t* wsb = p.w_scales + n0 * knb;
  const int xlast = (int)min(p.M - m0, (int64_t)BM) - 1, wlast = (int)min(p.N - n0, (int64_t)BN) - 1;
  auto scale_row = [&](int i) {
    return 64 * i < BM ? xsb + (uint32_t)min(srow + 64 * i, xlast) * (uint32_t)knb
                       : wsb + (uint32_t)min(srow + 64 * i - BM, wlast) * (uint32_t)knb;
  };
  auto load_scales = [&](int grp) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const uint8_t* row = scale_row(i);
      __builtin_memcpy(&sreg[i], row + mx4_scale_at(kp, grp, quarter), 16);  // at any alignment
    }
  };
  auto store_scales = [&](int pair) {  // of stages 2 pair and 2 pair + 1
    if (pair * 16 + 16 > nb && knb >= 16) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) sreg[i] = mx4_cut_scales(sreg[i], 16u - ((uint32_t)nb & 15u));
    }
    if (quarter == (pair & 3)) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) *(u32x4*)&sm.sc[pair & 1][(srow + 64 * i) * 16] = sreg[i];
    }
  };

  floatx16 acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int g = 0; g < FM; ++g)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][g][v] = 0.0f;

  u32x4 wf[2][FN], xf[2][FM];       // fragments of two steps
  int wsc[FN], xsc[FM], wnx[FN], xnx[FM];  // scale words of this stage and the next
  int slot[4];                      // lane's byte within a 32-row group, by step
#pragma unroll
  for (int s = 0; s < 4; ++s) slot[s] = r32 * 128 + 16 * ((4 * h + s) ^ x_swz(r32));
  // fragment f of step s in the order the MFMAs need them: w0, x0 .. x(FM-1), w1, ..
  auto read_frag = [&](int f, int s, int par, int buf) {
    const bool is_w = f == 0 || f > FM;
    const int idx = f == 0 ? 0 : (f <= FM ? f - 1 : f - FM);
    if (is_w) wf[par][idx] = *(const u32x4*)&sm.w[buf][(wave_n * FN + idx) * 4096 + slot[s]];
    else xf[par][idx] = *(const u32x4*)&sm.x[buf][(wave_m * FM + idx) * 4096 + slot[s]];
  };
  auto read_scales = [&](int stage, int (&w)[FN], int (&x)[FM]) {
    const uint8_t* sc = &sm.sc[(stage >> 1) & 1][8 * (stage & 1) + 4 * h];
#pragma unroll
    for (int i = 0; i < FN; ++i) w[i] = *(const int*)&sc[(BM + wave_n * WTN + i * 32 + r32) * 16];
#pragma unroll
    for (int g = 0; g < FM; ++g) x[g] = *(const int*)&sc[(wave_m * WTM + g * 32 + r32) * 16];
  };
  auto mfma = [&](int q, auto step) {
    constexpr int s = decltype(step)::value;
    const int i = q / FM, g = q % FM;
    const u32x4 a = wf[s & 1][i], b = xf[s & 1][g];
    const v8i_t av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
    const v8i_t bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
    acc[i][g] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, acc[i][g], 4, 4, s, wsc[i], s, xsc[g]);
  };

  // prologue: scale group 0, stages 0 .. NBUF - 2 and scale group 1; then stage 0's first step
  if (KS > 1 || knb >= 16) {
    load_scales(0);
  } else {  // a row of fewer than 16 scale bytes: byte by byte
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const uint8_t* row = scale_row(i);
      uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int b = 0; b < 15; ++b) {
        const uint32_t byte = row[min(b, knb - 1)];
        w[b >> 2] |= (b < knb ? byte : 0u) << (8 * (b & 3));
      }
      sreg[i] = u32x4{w[0], w[1], w[2], w[3]};
    }
  }
#pragma unroll
  for (int j = 0; j < kLoads; ++j) issue_code(j, 0, 0);
  store_scales(0);
#pragma unroll
  for (int b = 1; b < NBUF; ++b)
#pragma unroll
    for (int j = 0; j < (b == NBUF - 1 ? kL3 : kLoads); ++j) issue_code(j, b, b);
  __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0), lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  read_scales(0, wsc, xsc);
#pragma unroll
  for (int f = 0; f < kFrags; ++f) read_frag(f, 0, 0, 0);

  // Stages past the last are asked for all the same: their loads lie past every window and
  // touch no memory, and what is read of them is not used.
  int buf = 0;
#pragma clang loop unroll(disable)
  for (int t = 0; t < nst; ++t) {
    // the next scale group's way through the registers, ahead of the stage: the stage itself
    // has to stay one basic block, or its MFMAs are moved behind the barrier
    if ((t & 7) == 6) {
      if (t + 2 < nst) load_scales((t >> 3) + 1);
    } else if ((t & 1) == 1) {
      if (t + 1 < nst) store_scales((t + 1) >> 1);
    }
    auto step = [&](auto sc_) {
      constexpr int s = decltype(sc_)::value;
#pragma unroll
      for (int q = 0; q < kMfma; ++q) {
        mfma(q, sc_);
#pragma unroll
        for (int f = q * kFrags / kMfma; f < (q + 1) * kFrags / kMfma; ++f) read_frag(f, s + 1, (s + 1) & 1, buf);
        if constexpr (s == 0) {
#pragma unroll
          for (int l = kL3 + q * (kL0 - kL3) / kMfma; l < kL3 + (q + 1) * (kL0 - kL3) / kMfma; ++l) issue_code(l, t - 1 + NBUF, buf == 0 ? NBUF - 1 : buf - 1);
        } else if constexpr (s == 1) {
#pragma unroll
          for (int l = kL0 + q * (kL1 - kL0) / kMfma; l < kL0 + (q + 1) * (kL1 - kL0) / kMfma; ++l) issue_code(l, t - 1 + NBUF, buf == 0 ? NBUF - 1 : buf - 1);
        } else {
#pragma unroll
          for (int l = kL1 + q * (kLoads - kL1) / kMfma; l < kL1 + (q + 1) * (kLoads - kL1) / kMfma; ++l) issue_code(l, t - 1 + NBUF, buf == 0 ? NBUF - 1 : buf - 1);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 1>{});
    step(std::integral_constant<int, 2>{});
    const int nbuf = buf + 1 == NBUF ? 0 : buf + 1;
    constexpr std::integral_constant<int, 3> last{};
#pragma unroll
    for (int q = 0; q < kHalf; ++q) {
      mfma(q, last);
      __builtin_amdgcn_sched_barrier(0);
    }
    // this wave's loads of stage t + 1 landed, and its reads of stage t
    __builtin_amdgcn_s_waitcnt(0x0070 | (kWait & 15) | ((kWait >> 4) << 14));
    __builtin_amdgcn_s_barrier();
    read_scales(t + 1, wnx, xnx);
    constexpr int kTail = kMfma - kHalf;
#pragma unroll
    for (int q = kHalf; q < kMfma; ++q) {
      mfma(q, last);
      const int u = q - kHalf;
#pragma unroll
      for (int l = u * kL3 / kTail; l < (u + 1) * kL3 / kTail; ++l) issue_code(l, t + NBUF, buf);
#pragma unroll
      for (int f = u * kFrags / kTail; f < (u + 1) * kFrags / kTail; ++f) read_frag(f, 0, 0, nbuf);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int i = 0; i < FN; ++i) wsc[i] = wnx[i];
#pragma unroll
    for (int g = 0; g < FM; ++g) xsc[g] = xnx[g];
    buf = nbuf;
  }

  __builtin_amdgcn_s_waitcnt(0x0070);
  __syncthreads();
  if constexpr (KS > 1) {
    static_assert(FN == 1 && FM == 1, "parts of K meet one block of 32 x 32 at a time");
    floatx16* sums = (floatx16*)&smem[0];  // [KS - 1][NW][64]
    static_assert((KS - 1) * NW * 64 * sizeof(floatx16) <= sizeof(smem), "the parts' sums fit");
    if (part > 0) sums[((part - 1) * NW + wave) * 64 + lane] = acc[0][0];
    __syncthreads();
    if (part > 0) return;
#pragma unroll
    for (int k = 1; k < KS; ++k) acc[0][0] += sums[((k - 1) * NW + wave) * 64 + lane];
  }
  constexpr int kArea = 32 * kStoreRowPad(FN);
  static_assert(NW * kArea * 2 <= sizeof(sm), "store staging fits");
  // (with KS > 1 a wave's staging area lies over sums that other waves read)
  uint16_t* area = (uint16_t*)&smem[0] + (KS > 1 ? (KS - 1) * NW * 64 * 32 : 0) + wave * kArea;
  static_assert(KS == 1 || (KS - 1) * NW * 64 * 64 + NW * kArea * 2 <= (int)sizeof(smem), "beside the sums");
  mx4_store_tile<FM, FN>(acc, p, m0 + wave_m * WTM, n0 + wave_n * WTN, lane, area);
}

// ---- GEMM, few activation rows --------------------------------------------------------
//
// At most 16 FB activation rows: bound by the weights' read, which has to be spread over the
// whole chip and to be in flight at once. A workgroup takes 16 FA weight rows; its NW waves take groups of 256 elements of
// K in turn (a 128-byte line of codes per row) straight into registers, kU groups at a time
// with the next kU in flight, and meet in LDS at the end. v_mfma_scale_f32_16x16x128_f8f6f4:
// lane (q, r) = (lane / 16, lane % 16) holds the 32 elements of row r's block q of a step and
// that block's scale. A lane takes blocks 2q and 2q + 1 of a group (32 contiguous bytes) in
// two steps, so that a load touches one line per row.
//
// The scale bytes of all the workgroup's rows are staged in LDS first, under the first loads
// of codes: one wide read per row at any alignment instead of a byte at a time.
//
// kFused: the activations come as bf16 and are quantized by every workgroup into its LDS
// (the first one also stores them to the workspace): no second launch, for a few rows.
NVFP4_HD int mx4_scale_pitch(int nb) { return ((nb + 7) & ~7) + 8; }

struct Mx4Quant {
  const u32x4* x;      // bf16 activations [M, K]
  uint32_t* packed;    // workspace: codes [M, K/2]
  uint8_t* scales;     // [M, K/32]
};

template <int NW, int FA, int FB, bool kFused>
__global__ void __launch_bounds__(64 * NW) gemm_mx4_rows_kernel(GemmProblem p, Mx4Quant fq) {
  extern __shared__ __align__(16) uint8_t lds[];
  constexpr int kU = 2;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, r = lane & 15;
  const int nb = (int)(p.K >> 5), ng = (nb + 7) >> 3;
  const uint32_t pitch = (uint32_t)p.K >> 1;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * FA);
  const int rows = (int)min(p.N - n0, (int64_t)(16 * FA));
  const int M = (int)p.M;
  const int sp = mx4_scale_pitch(nb);
  uint8_t* wsc = lds;                        // [16 FA][sp]
  uint8_t* xsc = lds + 16 * FA * sp;         // [16 FB][sp]
  uint8_t* xq = xsc + 16 * FB * sp;          // kFused: [M][pitch + 16]
  const uint32_t xp = pitch + 16;

  const __amdgpu_buffer_rsrc_t rw = window_rsrc(p.w_packed, n0, n0 + rows, pitch);
  const __amdgpu_buffer_rsrc_t rx = kFused ? rw : window_rsrc(p.a_packed, 0, M, pitch);
  struct Group {
    u32x4 w[FA][2], x[FB][2];
  };
  auto load = [&](Group& g, int at) {
    // blocks past K (and groups past the last) lie past every window: zeros, no access
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int a = 0; a < FA; ++a)
        g.w[a][i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
            rw, (int)mx4_rows_voff(min(16 * a + r, rows - 1), q, i, at, nb, pitch), at * 128, 0));
      if constexpr (!kFused) {
#pragma unroll
        for (int b = 0; b < FB; ++b)
          g.x[b][i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
              rx, (int)mx4_rows_voff(min(16 * b + r, M - 1), q, i, at, nb, pitch), at * 128, 0));
      }
    }
  };
  Group cur[kU], nxt[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) load(cur[u], wave + u * NW);

  // scale bytes: a dword per lane, a wave's rows at once
  auto stage_scales = [&](const uint8_t* from, uint8_t* to, int n, auto frags) {
    constexpr int kPer = (16 * decltype(frags)::value + NW - 1) / NW;
    for (int at = 4 * lane; at < nb; at += 256) {
      uint32_t v[kPer];
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const uint8_t* src = from + (int64_t)min(wave + j * NW, n - 1) * nb + at;
        if (at + 4 <= nb) {
          __builtin_memcpy(&v[j], src, 4);
        } else {
          v[j] = src[0];
          if (at + 1 < nb) v[j] |= (uint32_t)src[1] << 8;
          if (at + 2 < nb) v[j] |= (uint32_t)src[2] << 16;
        }
      }
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (wave + j * NW < n) *(uint32_t*)&to[(wave + j * NW) * sp + at] = v[j];
    }
  };
  stage_scales(p.w_scales + n0 * nb, wsc, rows, std::integral_constant<int, FA>{});
  if constexpr (kFused) {
    // as mx4_quantize_kernel: four threads to a block, eight elements each
    const int per = (int)(p.K >> 3), n = M * per;
    for (int i = threadIdx.x; i < n; i += 64 * NW) {  // n is a multiple of 4: quads stay whole
      const Mx4Codes c = mx4_encode_quad(fq.x[i]);
      const int row = i / per, at = i - row * per;
      *(uint32_t*)&xq[row * xp + 4 * at] = c.word;
      if ((i & 3) == 0) xsc[row * sp + (at >> 2)] = (uint8_t)c.byte;
      if (blockIdx.x == 0) {
        fq.packed[i] = c.word;
        if ((i & 3) == 0) fq.scales[i >> 2] = (uint8_t)c.byte;
      }
    }
  } else {
    stage_scales(p.a_scales, xsc, M, std::integral_constant<int, FB>{});
  }
  __syncthreads();

  floatx4 acc[FA][FB];
#pragma unroll
  for (int a = 0; a < FA; ++a)
#pragma unroll
    for (int b = 0; b < FB; ++b) acc[a][b] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  int ws[FA], xs[FB];  // offsets of this lane's rows in the staged scales
#pragma unroll
  for (int a = 0; a < FA; ++a) ws[a] = min(16 * a + r, rows - 1) * sp + 2 * q;
#pragma unroll
  for (int b = 0; b < FB; ++b) xs[b] = min(16 * b + r, M - 1) * sp + 2 * q;
  auto multiply = [&](const Group& g, int at) {
    if (at >= ng) return;
    // (bytes past nb in the padded rows are whatever LDS held: their lanes take zero codes, and
    // a scale that may be NaN must not meet them)
    const bool in0 = 8 * at + 2 * q < nb, in1 = 8 * at + 2 * q + 1 < nb;
    int sw[FA], sx[FB];
#pragma unroll
    for (int a = 0; a < FA; ++a) sw[a] = *(const uint16_t*)&wsc[ws[a] + 8 * at];
#pragma unroll
    for (int b = 0; b < FB; ++b) sx[b] = *(const uint16_t*)&xsc[xs[b] + 8 * at];
    const int mask = in1 ? 0xFFFF : in0 ? 0xFF : 0;
#pragma unroll
    for (int a = 0; a < FA; ++a) sw[a] &= mask;
#pragma unroll
    for (int b = 0; b < FB; ++b) sx[b] &= mask;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v8i_t av[FA], bv[FB];
#pragma unroll
      for (int a = 0; a < FA; ++a) {
        const u32x4 c = g.w[a][i];
        av[a] = v8i_t{(int)c.x, (int)c.y, (int)c.z, (int)c.w, 0, 0, 0, 0};
      }
#pragma unroll
      for (int b = 0; b < FB; ++b) {
        u32x4 c;
        if constexpr (kFused) {
          c = (i == 0 ? in0 : in1) ? *(const u32x4*)&xq[(uint32_t)min(16 * b + r, M - 1) * xp + 128u * (uint32_t)at + 32u * (uint32_t)q + 16u * i] : u32x4{0u, 0u, 0u, 0u};
        } else {
          c = g.x[b][i];
        }
        bv[b] = v8i_t{(int)c.x, (int)c.y, (int)c.z, (int)c.w, 0, 0, 0, 0};
      }
#pragma unroll
      for (int a = 0; a < FA; ++a)
#pragma unroll
        for (int b = 0; b < FB; ++b) {
          if (i == 0)
            acc[a][b] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av[a], bv[b], acc[a][b], 4, 4, 0, sw[a], 0, sx[b]);
          else
            acc[a][b] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av[a], bv[b], acc[a][b], 4, 4, 1, sw[a], 1, sx[b]);
        }
    }
  };
  for (int g = wave; g < ng; g += kU * NW) {
    const bool more = g + kU * NW < ng;
    if (more) {
#pragma unroll
      for (int u = 0; u < kU; ++u) load(nxt[u], g + (kU + u) * NW);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) multiply(cur[u], g + u * NW);
    if (more) {
#pragma unroll
      for (int u = 0; u < kU; ++u) cur[u] = nxt[u];
    }
  }

  // the waves' sums meet in LDS (over the staged scales) in wave order
  __syncthreads();
  floatx4* part = (floatx4*)lds;  // [NW][FA][FB][64]
#pragma unroll
  for (int a = 0; a < FA; ++a)
#pragma unroll
    for (int b = 0; b < FB; ++b) part[((wave * FA + a) * FB + b) * 64 + lane] = acc[a][b];
  __syncthreads();
  for (int i = threadIdx.x; i < FA * FB * 64; i += 64 * NW) {
    floatx4 v = part[i];
#pragma unroll
    for (int w = 1; w < NW; ++w) v += part[w * FA * FB * 64 + i];
    const int l = i & 63, f = i >> 6, a = f / FB, b = f % FB;
    const int m = 16 * b + (l & 15), n = 16 * a + 4 * (l >> 4);
    if (m < M && n < rows) {
      uint16_t* o = p.out + (int64_t)m * p.N + n0 + n;
      const u32x2 w = bf16x4_rne(v[0], v[1], v[2], v[3]);
      if (n + 3 < rows) {
        __builtin_memcpy(o, &w, 8);
      } else {
        for (int e = 0; n + e < rows; ++e) o[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
      }
    }
  }
}

}  // namespace

namespace {

// LDS of the kernel for few rows: the staged scales, or the waves' sums that follow them.
int64_t mx4_rows_lds(int64_t M, int64_t K) {
  const int64_t pitch = mx4_scale_pitch((int)(K >> 5));
  const int64_t fb = M <= 16 ? 1 : M <= 32 ? 2 : 4, fa = fb == 2 ? 2 : 1, waves = fb == 1 ? 16 : 8;
  const int64_t scales = 16 * (fa + fb) * pitch, sums = waves * fa * fb * 1024;
  return scales > sums ? scales : sums;
}

template <int NW, int FA, int FB, bool kFused>
void launch_rows(const GemmProblem& p, const Mx4Quant& fq, size_t lds, hipStream_t stream) {
  hipLaunchKernelGGL((gemm_mx4_rows_kernel<NW, FA, FB, kFused>), dim3((unsigned)((p.N + 16 * FA - 1) / (16 * FA))),
                     dim3(64 * NW), lds, stream, p, fq);
}

}  // namespace

hipError_t launch_mx4_quantize(const void* x, int64_t M, int64_t K, void* packed, void* scales,
                               hipStream_t stream, const LaunchInfo& dev) {
  const int64_t nlanes = M * K / 8;
  if (nlanes == 0) return hipSuccess;
  constexpr int kThreads = 256, kUnroll = 2;
  const int64_t want = (nlanes + (int64_t)kThreads * kUnroll - 1) / ((int64_t)kThreads * kUnroll);
  const int64_t cap = (int64_t)dev.num_cus * 32;
  hipLaunchKernelGGL((mx4_quantize_kernel<kUnroll>), dim3((unsigned)(want < cap ? want : cap)),
                     dim3(kThreads), 0, stream, (const u32x4*)x, (uint32_t*)packed,
                     (uint8_t*)scales, nlanes);
  return hipGetLastError();
}

hipError_t launch_mx4_dequantize(const void* packed, const void* scales, int64_t M, int64_t K,
                                 void* out, hipStream_t stream, const LaunchInfo& dev) {
  const int64_t nlanes = M * K / 8;
  if (nlanes == 0) return hipSuccess;
  constexpr int kThreads = 256, kUnroll = 2;
  const int64_t want = (nlanes + (int64_t)kThreads * kUnroll - 1) / ((int64_t)kThreads * kUnroll);
  const int64_t cap = (int64_t)dev.num_cus * 32;
  hipLaunchKernelGGL((mx4_dequantize_kernel<kUnroll>), dim3((unsigned)(want < cap ? want : cap)),
                     dim3(kThreads), 0, stream, (const uint32_t*)packed, (const uint8_t*)scales,
                     (u32x4*)out, nlanes);
  return hipGetLastError();
}

// ---- which kernel ---------------------------------------------------------------------

namespace {

// One tiling of the product. Times in microseconds, fitted to launches of one to eight passes
// at K = 4096 and 8192: a pass of one workgroup per compute unit takes base + stages * alone;
// where a compute unit holds two workgroups (or, for the 256 x 256 tile, where the whole chip
// multiplies and its clock falls) base + stages * together. ragged: what the stores of a
// width that is no multiple of 8 add.
struct Mx4Tile {
  int kernel, bm, bn, resident;
  float base, ragged, alone, together;
};
constexpr Mx4Tile kMx4Tiles[] = {
    {NVFP4_MXFP4_TILE256, 256, 256, 1, 3.5f, 8.0f, 1.5f, 2.1f},
    {NVFP4_MXFP4_TILE128X256, 128, 256, 1, 4.8f, 4.0f, 0.94f, 1.25f},
    {NVFP4_MXFP4_TILE128, 128, 128, 2, 2.0f, 1.5f, 0.72f, 1.3f},
    {NVFP4_MXFP4_TILE64X128, 64, 128, 2, 1.2f, 0.8f, 0.5f, 0.84f},
    {NVFP4_MXFP4_TILE64, 64, 64, 2, 1.3f, 0.3f, 0.43f, 0.46f},
};

constexpr int64_t kMx4MaxTiles = (1 << 24) - 1;  // a launch has fewer than 2^32 threads

}  // namespace

// * Few rows: the kernel for them, while its staged scales fit its LDS and one or two passes
//   of its workgroups cover the weight rows (17 x 14336 x 4096: 10.3 us against 8.2 with 64 x
//   64 tiles; 33 x 4012 x 5760: 8.2 against 10.2; 33 x 1000 x 2880: 5.1 against 6.7; 48 x 6144 x
//   4096: 9.8 against 7.9).
// * Else the tiling of least estimated time. Products that one pass of 64 x 64 tiles covers
//   split a long K over two halves of the workgroup (256 x 4096 x 4096: 8.1 us against 9.8; 500
//   x 2048 x 2048: 5.9 against 6.5; but 344 x 710 x 768: 4.6 against 4.3; its scale reads need
//   K > 1024).
int plan_mx4_gemm(int64_t M, int64_t N, int64_t K, int64_t cus) {
  if (cus <= 0) cus = 256;
  if (mx4_rows_lds(M, K) <= 65536 && ((M <= 32 && N <= 32 * cus) || (M <= 40 && N <= 16 * cus) ||
                                      (M <= 64 && N <= 4 * cus && K <= 4096)))
    return NVFP4_MXFP4_ROWS;
  const int64_t t64 = ((M + 63) / 64) * ((N + 63) / 64);
  if (t64 <= cus && K > 1024 && mx4_parts_ok((int)(K >> 5), 2)) return NVFP4_MXFP4_SPLIT64;
  const float stages = (float)((K + 255) / 256);
  int best = 0;
  float least = 0.0f;
  for (const Mx4Tile& t : kMx4Tiles) {
    const int64_t tiles = ((M + t.bm - 1) / t.bm) * ((N + t.bn - 1) / t.bn);
    if (best != 0 && tiles > kMx4MaxTiles) continue;  // (the largest tile comes first)
    const int64_t load = (tiles + cus - 1) / cus;  // tiles of the busiest compute unit
    const float base = t.base + (N % 8 != 0 ? t.ragged : 0.0f);
    float us;
    if (t.resident == 2) {
      us = (float)(load / 2) * (base + stages * t.together) + (float)(load % 2) * (base + stages * t.alone);
    } else {
      const float fill = load > 1 ? 1.0f : (float)tiles / (float)cus;
      us = (float)load * (base + stages * (t.alone + fill * (t.together - t.alone)));
    }
    if (best == 0 || us < least) {
      best = t.kernel;
      least = us;
    }
  }
  return best;
}

Mx4Form mx4_form(int64_t M, int64_t N, int64_t K, int64_t cus) {
  if (cus <= 0) cus = 256;
  const int kernel = plan_mx4_gemm(M, N, K, cus);
  switch (kernel) {
    case NVFP4_MXFP4_ROWS:
      // 16 waves for a long K (8 waves against 16, launches in a graph, weights past the caches: 1 x 4096
      // x 8192 7.8 us / 6.5, 1 x 8192 x 8192 11.5 / 10.8, 1 x 4096 x 14336 10.2 / 9.9, though 1 x 5120 x
      // 14336 14.5 / 16.1; 1 x 4096 x 7168 6.8 / 6.2, 1 x 8192 x 7168 9.7 / 10.2, 1 x 4096 x 4096
      // 4.9 / 5.4, 1 x 8192 x 4096 6.4 / 8.6); two weight fragments where one would take a second pass
      if (M <= 16) return Mx4Form{kernel, 16, 16, K >= 8192 ? 16 : 8};
      if (M <= 32) return Mx4Form{kernel, 32, N <= 16 * cus ? 16 : 32, 8};
      return Mx4Form{kernel, 64, 16, 8};
    case NVFP4_MXFP4_SPLIT64: return Mx4Form{kernel, 64, 64, 3};
    case NVFP4_MXFP4_TILE64: return Mx4Form{kernel, 64, 64, 4};
    case NVFP4_MXFP4_TILE64X128: return Mx4Form{kernel, 64, 128, 3};
    case NVFP4_MXFP4_TILE128:
      // one workgroup per compute unit: loads four stages ahead (1024 x 4096 x 4096: 16.2 us
      // against 17.5 with two); more tiles: two workgroups per compute unit (4096 x 4096 x 4096:
      // 48 against 55 us)
      return Mx4Form{kernel, 128, 128, ((M + 127) / 128) * ((N + 127) / 128) <= cus ? 4 : 2};
    case NVFP4_MXFP4_TILE128X256: return Mx4Form{kernel, 128, 256, 3};
    default: return Mx4Form{kernel, 256, 256, 2};
  }
}

hipError_t launch_mx4_gemm(const GemmProblem& p, hipStream_t stream, const LaunchInfo& dev) {
  auto tiles = [&](int64_t bm, int64_t bn) { return ((p.M + bm - 1) / bm) * ((p.N + bn - 1) / bn); };
  if (tiles(256, 256) > kMx4MaxTiles) return hipErrorInvalidValue;
#define NVFP4_MX4_TILE(BM, BN, NBUF, KS)                                                              \
  hipLaunchKernelGGL((gemm_mx4_kernel<BM, BN, NBUF, KS>), dim3((unsigned)tiles(BM, BN)), dim3(256 * KS), 0, \
                     stream, p)
  const Mx4Form f = mx4_form(p.M, p.N, p.K, dev.num_cus);
  switch (f.kernel) {
    case NVFP4_MXFP4_ROWS: {
      const size_t lds = (size_t)mx4_rows_lds(p.M, p.K);
      if (f.m == 16) {
        if (f.depth == 16) launch_rows<16, 1, 1, false>(p, Mx4Quant{}, lds, stream);
        else launch_rows<8, 1, 1, false>(p, Mx4Quant{}, lds, stream);
      } else if (f.m == 32) {
        if (f.n == 16) launch_rows<8, 1, 2, false>(p, Mx4Quant{}, lds, stream);
        else launch_rows<8, 2, 2, false>(p, Mx4Quant{}, lds, stream);
      } else {
        launch_rows<8, 1, 4, false>(p, Mx4Quant{}, lds, stream);
      }
      break;
    }
    case NVFP4_MXFP4_SPLIT64: NVFP4_MX4_TILE(64, 64, 3, 2); break;
    case NVFP4_MXFP4_TILE64: NVFP4_MX4_TILE(64, 64, 4, 1); break;
    case NVFP4_MXFP4_TILE64X128: NVFP4_MX4_TILE(64, 128, 3, 1); break;
    case NVFP4_MXFP4_TILE128:
      if (f.depth == 4) NVFP4_MX4_TILE(128, 128, 4, 1);
      else NVFP4_MX4_TILE(128, 128, 2, 1);
      break;
    case NVFP4_MXFP4_TILE128X256: NVFP4_MX4_TILE(128, 256, 3, 1); break;
    default: NVFP4_MX4_TILE(256, 256, 2, 1); break;
  }
#undef NVFP4_MX4_TILE
  return hipGetLastError();
}

bool mx4_linear_fused(int64_t M, int64_t N, int64_t K, int64_t cus) {
  return M > 0 && N > 0 && M <= 16 && M * K <= 24576 && plan_mx4_gemm(M, N, K, cus) == NVFP4_MXFP4_ROWS &&
         mx4_rows_lds(M, K) + M * (K / 2 + 16) <= 65536;
}

hipError_t launch_mx4_linear_fused(const GemmProblem& p, const void* x, void* packed, void* scales,
                                   hipStream_t stream) {
  const Mx4Quant fq{(const u32x4*)x, (uint32_t*)packed, (uint8_t*)scales};
  const size_t lds = (size_t)(mx4_rows_lds(p.M, p.K) + p.M * (p.K / 2 + 16));
  if (p.K >= 8192) launch_rows<16, 1, 1, true>(p, fq, lds, stream);  // (as without: mx4_form)
  else launch_rows<8, 1, 1, true>(p, fq, lds, stream);
  return hipGetLastError();
}

}  // namespace nvfp4
