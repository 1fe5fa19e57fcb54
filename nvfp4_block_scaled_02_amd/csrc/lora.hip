// Low-rank adapters of many requests beside a shared projection, for gfx950.
//
// For row t with adapter a = adapters[t] in [0, L):
//   v_t = s_a * A_a x_t  (R sums over K),   out_t = bf16(y_t + B_a v_t);
// any other row keeps y_t. x [T, K], A [L, R, K], B [L, N, R], y and out [T, N], all bf16.
//
// Two kernels, the product with A and that with B. Both work on tiles of 16 rows with
// v_mfma_f32_16x16x32_bf16: the adapter's rows are its A operand, 16 rows of activations its
// columns, so that a result column belongs to one row alone. Rows come in any order: a workgroup
// lists the distinct adapters of its rows, takes them one after the other and keeps of each result
// the columns whose adapter it is. Where there are few rows the adapters are dealt out to several
// workgroups (grid z) instead.
//
// Between the products v keeps its 32 bits: the matrix instruction takes bf16, so v goes in as three
// bf16 parts that add up to it. (Two, 2^-16 of it, turn the rounding of 3 outputs in a thousand from
// what fp32 gives, three of 2 in ten thousand, as any other order of the sums does; the third takes
// 0 to 3 % of both products' time: 1999 rows of rank 64 into 14336 54.6 us instead of 53.0, 16384 rows of
// rank 16 into 4096 86.1 instead of 84.9.)
#include "gemm_common.hpp"
#include "lora_offsets.hpp"

namespace nvfp4 {

namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

__device__ __forceinline__ floatx4 mfma(const u32x4 a, const u32x4 b, const floatx4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b),
                                                 c, 0, 0, 0);
}

// A row's adapter, -1 where it has none.
__device__ __forceinline__ int adapter_of(const LoraProblem& p, int64_t t) {
  const int a = t < p.T ? p.adapters[t] : -1;
  return a >= 0 && a < p.L ? a : -1;
}

// Calls f(adapter) for the distinct adapters of the lanes that are this workgroup's: the i-th
// where i % gridDim.z == blockIdx.z.
template <typename F>
__device__ __forceinline__ void for_adapters(int adapter, const F& f) {
  uint64_t left = __ballot(adapter >= 0);
  for (unsigned i = 0; left != 0; ++i) {
    const int a = __builtin_amdgcn_readlane(adapter, __builtin_ctzll(left));
    left &= ~__ballot(adapter == a);
    if (i % gridDim.z == blockIdx.z) f(a);
  }
}

// Four values in three bf16 parts each: 8 bits of a value (cut, so that they overflow with the value
// alone), 8 of the rest, and what is left, which has 8 at most: their sum is the value itself (below
// 2^-109, where bits of the last part are below the least bf16, within 2^-134). An infinity has no rest.
struct Parts {
  u32x2 of[3];
};
__device__ __forceinline__ Parts three_parts(const floatx4 v) {
  float rest[4];
  uint32_t b[4], m[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    b[j] = f2u(v[j]);
    rest[j] = (b[j] & 0x7FFFFFFFu) == 0x7F800000u ? 0.0f : v[j] - u2f(b[j] & 0xFFFF0000u);
    m[j] = f2u(rest[j]);
    rest[j] -= u2f(m[j] & 0xFFFF0000u);
  }
  return Parts{{u32x2{(b[0] >> 16) | (b[1] & 0xFFFF0000u), (b[2] >> 16) | (b[3] & 0xFFFF0000u)},
                u32x2{(m[0] >> 16) | (m[1] & 0xFFFF0000u), (m[2] >> 16) | (m[3] & 0xFFFF0000u)},
                bf16x4_rne(rest[0], rest[1], rest[2], rest[3])}};
}

// ---- v = s A x, 16 rows ----
//
// A workgroup's waves take units of 8 kC elements of K in turn, each for itself. A unit comes through
// LDS (16 kC consecutive bytes of a row, 64 / kC rows per load): loaded in the matrix instruction's
// order, every load touches 16 rows and takes half as long again (16384 rows of K 4096 and rank 16, 34 us
// as it is) to twice as long (1999 of rank 64, 13). Chunk c (16 bytes) of row s sits at slot
// c ^ (s % 16), so that the 16 rows of a fragment read are in distinct banks.
template <int kR, int kC>
constexpr int kUnitBytes = (1 + kR) * 16 * 16 * kC;
// acc: this wave's share, of kR fragments of 16 ranks from A's row at w on.
template <int kR, int kC, int kWaves>
__device__ __forceinline__ void down_units(floatx4 (&acc)[kR], __amdgpu_buffer_rsrc_t rx, __amdgpu_buffer_rsrc_t rw, uint32_t pitch,
                                           int chunks, int wave, int lane, uint8_t* mine) {
  constexpr int kRowBytes = 16 * kC, kTileBytes = 16 * kRowBytes;
  const int q = lane >> 4, r = lane & 15, units = (chunks + kC - 1) / kC;
#pragma unroll
  for (int i = 0; i < kR; ++i) acc[i] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int u = wave; u < units; u += kWaves) {
#pragma unroll
    for (int i = 0; i < 1 + kR; ++i)
#pragma unroll
      for (int k = 0; k < kC / 4; ++k)
        buffer_load_lds16(i == 0 ? rx : rw, mine + i * kTileBytes + 1024 * k,
                          lora_stage_voff<kC>(lane, k, i == 0 ? 0 : 16 * (i - 1), pitch, u, chunks), (uint32_t)(u * kRowBytes));
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int k = 0; k < kC / 4; ++k) {
      const int at = r * kRowBytes + 16 * ((4 * k + q) ^ r);
      const u32x4 x = *(const u32x4*)&mine[at];
#pragma unroll
      for (int i = 0; i < kR; ++i) acc[i] = mfma(*(const u32x4*)&mine[(1 + i) * kTileBytes + at], x, acc[i]);
    }
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): read before the next unit comes
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  }
}
// Windows of 16 rows of x from t0 on and of `ranks` rows of A from adapter a's r0 on; rows past them
// read as zero.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t x_window(const LoraProblem& p, int64_t t0, int rows) {
  return make_rsrc(p.x + t0 * p.K, (uint32_t)min(p.T - t0, (int64_t)rows) * (uint32_t)(p.K * 2));
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t a_window(const LoraProblem& p, int a, int r0, int rows) {
  return make_rsrc(p.a + ((int64_t)a * p.R + r0) * p.K, (uint32_t)min(p.R - r0, rows) * (uint32_t)(p.K * 2));
}
// The waves' shares of fragment i, added in their order; `part` holds [wave][kR][64].
template <int kR, int kWaves>
__device__ __forceinline__ floatx4 down_sum(const floatx4* part, int i, int lane) {
  floatx4 v = part[i * 64 + lane];
#pragma unroll
  for (int n = 1; n < kWaves; ++n) v += part[(n * kR + i) * 64 + lane];
  return v;
}
// Four ranks of row r's v, scaled, in its parts: to chunks of a tile (lora_chunk), as the second product
// loads them: a chunk's 16 rows together, so that 64 lanes load 1024 consecutive bytes (row by row each
// lane would meet a line of its own: 8192 rows of rank 64 into 4096 45 us instead of 39).
__device__ __forceinline__ void store_parts(u32x4* tile, int r, int rank, int R, const floatx4 v) {
  const Parts parts = three_parts(v);
#pragma unroll
  for (int i = 0; i < 3; ++i) ((u32x2*)&tile[(i * (R >> 3) + (rank >> 3)) * 16 + r])[(rank >> 2) & 1] = parts.of[i];
}
// Of a tile, the chunk that a lane takes in step k (where it has none: the first).
__device__ __forceinline__ u32x4 v_chunk(const u32x4* tile, int k, int steps, int R, int q, int r) {
  return tile[max(lora_chunk(k, q, steps, R), 0) * 16 + r];
}
// The chunks of a tile of 16 rows in the workspace.
__device__ __forceinline__ u32x4* v_tile(const LoraProblem& p, int64_t tile) {
  return (u32x4*)p.down + tile * lora_tile_chunks(p.R);
}

template <int kR, int kC, int kWaves>
__global__ void __launch_bounds__(64 * kWaves) lora_down_kernel(LoraProblem p) {
  constexpr int kBytes = kUnitBytes<kR, kC>;
  static_assert(kBytes >= kR * 1024, "the sums meet in the same memory");
  __shared__ __align__(16) uint8_t lds[kWaves * kBytes];
  const int lane = threadIdx.x & 63, q = lane >> 4, r = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const LoraPart part_of = lora_part(blockIdx.x, gridDim.x, p.R, 16 * kR);
  const int64_t t0 = part_of.tile * 16;
  const int r0 = part_of.rank;
  const int adapter = lane < 16 ? adapter_of(p, t0 + lane) : -1;
  const __amdgpu_buffer_rsrc_t rx = x_window(p, t0, 16);
  for_adapters(adapter, [&](int a) {
    floatx4 acc[kR];
    down_units<kR, kC, kWaves>(acc, rx, a_window(p, a, r0, 16 * kR), (uint32_t)(p.K * 2), (int)(p.K >> 3), wave, lane,
                               lds + wave * kBytes);
    __syncthreads();
    floatx4* part = (floatx4*)lds;
#pragma unroll
    for (int i = 0; i < kR; ++i) part[(wave * kR + i) * 64 + lane] = acc[i];
    __syncthreads();
    const float s = p.scales ? p.scales[a] : 1.0f;
    for (int i = wave; i < kR; i += kWaves) {
      const int rank = r0 + 16 * i + 4 * q;  // R % 8 == 0: four ranks are all there or none
      if (__shfl(adapter, r, 64) == a && rank < p.R)
        store_parts(v_tile(p, part_of.tile), r, rank, p.R, down_sum<kR, kWaves>(part, i, lane) * s);
    }
    __syncthreads();
  });
}

// The same for many rows: kTok tiles of 16 rows and kR fragments of 16 ranks per workgroup, whose
// kTok * kSplit waves stage both together, kBufs - 1 stages of 8 kC elements of K ahead; a wave multiplies
// one tile, of every kSplit steps of 32 elements one.
template <int kR, int kTok, int kSplit, int kC, int kBufs>
__global__ void __launch_bounds__(64 * kTok * kSplit) lora_down_wide_kernel(LoraProblem p) {
  constexpr int kWaves = kTok * kSplit, kRowBytes = 16 * kC, kTileBytes = 16 * kRowBytes;
  constexpr int kStage = (kTok + kR) * kTileBytes;
  constexpr int kLoads = kStage / 1024 / kWaves;  // of a wave and stage
  static_assert(kStage % (1024 * kWaves) == 0 && kC % (4 * kSplit) == 0, "whole turns");
  static_assert(kSplit == 1 || kBufs * kStage >= kWaves * kR * 1024, "the sums meet in the same memory");
  __shared__ __align__(16) uint8_t lds[kBufs * kStage];
  const int lane = threadIdx.x & 63, q = lane >> 4, r = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tile = wave % kTok, split = wave / kTok;
  const LoraPart part_of = lora_part(blockIdx.x, gridDim.x, p.R, 16 * kR);
  const int64_t t0 = part_of.tile * (16 * kTok);
  const int r0 = part_of.rank;
  const int adapter = lane < 16 * kTok ? adapter_of(p, t0 + lane) : -1;
  const int chunks = (int)(p.K >> 3), stages = (chunks + kC - 1) / kC;
  const uint32_t pitch = (uint32_t)(p.K * 2);
  const __amdgpu_buffer_rsrc_t rx = x_window(p, t0, 16 * kTok);
  for_adapters(adapter, [&](int a) {
    const __amdgpu_buffer_rsrc_t rw = a_window(p, a, r0, 16 * kR);
    floatx4 acc[kR];
#pragma unroll
    for (int i = 0; i < kR; ++i) acc[i] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    auto stage = [&](int u, int buf) {  // past the last stage: nothing is read, zeros are written
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int piece = i * kWaves + wave;  // of 64 / kC rows
        constexpr int kOfX = kTok * kC / 4;
        const bool of_x = piece < kOfX;
        buffer_load_lds16(of_x ? rx : rw, lds + buf * kStage + 1024 * piece,
                          lora_stage_voff<kC>(lane, of_x ? piece : piece - kOfX, 0, pitch, u, chunks), (uint32_t)(u * kRowBytes));
      }
    };
#pragma unroll
    for (int b = 0; b < kBufs - 1; ++b) stage(b, b);
    for (int u = 0, buf = 0; u < stages; ++u) {
      constexpr int kWait = (kBufs - 2) * kLoads;  // of later stages
      __builtin_amdgcn_s_waitcnt(0x0070 | (kWait & 15) | ((kWait >> 4) << 14));
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
      stage(u + kBufs - 1, buf == 0 ? kBufs - 1 : buf - 1);
      const uint8_t* at = lds + buf * kStage;
#pragma unroll
      for (int k = 0; k < kC / 4 / kSplit; ++k) {
        const int slot = r * kRowBytes + 16 * ((4 * (k * kSplit + split) + q) ^ r);
        const u32x4 x = *(const u32x4*)&at[tile * kTileBytes + slot];
#pragma unroll
        for (int i = 0; i < kR; ++i) acc[i] = mfma(*(const u32x4*)&at[(kTok + i) * kTileBytes + slot], x, acc[i]);
      }
      __builtin_amdgcn_sched_barrier(0);
      buf = buf + 1 == kBufs ? 0 : buf + 1;
    }
    __builtin_amdgcn_s_waitcnt(0x0070);
    __syncthreads();
    const float s = p.scales ? p.scales[a] : 1.0f;
    const bool here = __shfl(adapter, 16 * tile + r, 64) == a;
    auto store = [&](int i, const floatx4 v) {
      const int rank = r0 + 16 * i + 4 * q;
      if (here && rank < p.R) store_parts(v_tile(p, part_of.tile * kTok + tile), r, rank, p.R, v * s);
    };
    if constexpr (kSplit == 1) {
#pragma unroll
      for (int i = 0; i < kR; ++i) store(i, acc[i]);
    } else {
      floatx4* part = (floatx4*)lds;
#pragma unroll
      for (int i = 0; i < kR; ++i) part[(wave * kR + i) * 64 + lane] = acc[i];
      __syncthreads();
      for (int i = split; i < kR; i += kSplit) {
        floatx4 v = part[(tile * kR + i) * 64 + lane];
#pragma unroll
        for (int n = 1; n < kSplit; ++n) v += part[((n * kTok + tile) * kR + i) * 64 + lane];
        store(i, v);
      }
      __syncthreads();
    }
  });
}

// ---- out = y + B v ----
//
// 64 columns of the output per wave, as four fragments of 16 rows of B such that a lane's results are
// 16 consecutive columns of its row. kSteps: lora_steps, kHalves: lora_halves. The lower parts, kLast
// steps, multiply the fragments of the first steps again.
template <int kSteps, bool kHalves>
struct UpWeights {
  static constexpr int kW = kHalves ? kSteps / 2 : kSteps, kLast = (kSteps + 1) / 2, kAll = kSteps + kLast;
  u32x4 w[kW][4];
  __device__ __forceinline__ void load(const LoraProblem& p, int a, int64_t n0, int q, int r) {
    const int R8 = p.R >> 3;
    const u32x4* b = (const u32x4*)p.b + (int64_t)a * p.N * R8;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const u32x4* from = b + min(n0 + lora_column(r, i), p.N - 1) * R8;
#pragma unroll
      for (int k = 0; k < kW; ++k) {
        const int c = 4 * k + q;
        w[k][i] = from[c % R8];
        if (p.R % 16 != 0 && c >= 2 * R8) w[k][i] = u32x4{0u, 0u, 0u, 0u};
      }
    }
  }
  // sum = B v where `here` (v: the lane's chunks of all parts), else as it was
  __device__ __forceinline__ void multiply(floatx4 (&sum)[4], const u32x4* v, bool here, int R, int q) const {
    floatx4 acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < kAll; ++k) {
      const int step = k < kSteps ? k % kW : k - kSteps;
      const u32x4 x = here && lora_chunk(k, q, kSteps, R) >= 0 ? v[k] : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = mfma(w[step][i], x, acc[i]);
    }
    if (here) {
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[i] = acc[i];
    }
  }
};

// The sums pass through LDS, so that y is read and out written in whole pieces of 128 kWaves bytes of
// a row (each lane with the columns that the matrix instruction gives it: 16 rows in every access,
// 16384 x 4096 of rank 16 77 us instead of 63). A thread has 8 columns of two rows of a tile.
//
// kWhole: N is a multiple of 8, and the loads have no branch around them that would wait for them.
// kPassing: they leave the caches to v and B, as the stores do; where y is larger than these
// (both products, 16384 x 4096 of rank 16, 91.7 us, passing 86.3; 8192 x 4096 of rank 64 72.6, 66.4; but
// 4096 x 2048 of rank 32 19.9, 22.2).
enum class Rows { kAny, kWhole, kPassing };
template <int kWaves, Rows kRows>
struct UpRows {
  static constexpr bool kWhole = kRows != Rows::kAny;
  static constexpr int kPitch = 64 * kWaves + 4;  // floats
  const int row, column;
  const int64_t n;
  const int there;
  u32x4 y[2];
  __device__ __forceinline__ UpRows(const LoraProblem& p, int64_t first)
      : row((int)threadIdx.x / (8 * kWaves)), column(8 * ((int)threadIdx.x % (8 * kWaves))), n(first + column),
        there((int)max(min(p.N - n, (int64_t)8), (int64_t)0)) {}
  __device__ __forceinline__ void load(const LoraProblem& p, int64_t t0, uint32_t wanted) {  // a bit per row
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int m = row + 8 * i;
      const bool want = ((wanted >> m) & 1) != 0;
      if constexpr (kWhole) {  // (of what is not wanted, something that is there)
        const u32x4* from = (const u32x4*)(p.y + (want ? min(t0 + m, p.T - 1) : t0) * p.N + (there != 0 ? n : 0));
        y[i] = kRows == Rows::kPassing ? __builtin_nontemporal_load(from) : *from;
      } else if (want) {
        const uint16_t* from = p.y + min(t0 + m, p.T - 1) * p.N + n;
        if (there == 8) {
          __builtin_memcpy(&y[i], from, 16);  // at any alignment
        } else {
          uint16_t e[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) e[c] = c < there ? from[c] : (uint16_t)0;
          __builtin_memcpy(&y[i], e, 16);
        }
      }
    }
  }
  // A wave's sums, and behind a barrier the rows of `write` (a bit each); those of `none` keep y's bits.
  static __device__ __forceinline__ void put(float* s, const floatx4 (&sum)[4], int wave, int q, int r) {
#pragma unroll
    for (int i = 0; i < 4; ++i) *(floatx4*)&s[r * kPitch + 64 * wave + 16 * q + 4 * i] = sum[i];
  }
  __device__ __forceinline__ void store(const LoraProblem& p, const float* s, int64_t t0, uint32_t write, uint32_t none) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int m = row + 8 * i;
      const floatx4 s0 = *(const floatx4*)&s[m * kPitch + column], s1 = *(const floatx4*)&s[m * kPitch + column + 4];
      const uint32_t y0 = y[i].x, y1 = y[i].y, y2 = y[i].z, y3 = y[i].w;
      u32x4 o = {bf16x2_rne(u2f(y0 << 16) + s0[0], u2f(y0 & 0xFFFF0000u) + s0[1]),
                 bf16x2_rne(u2f(y1 << 16) + s0[2], u2f(y1 & 0xFFFF0000u) + s0[3]),
                 bf16x2_rne(u2f(y2 << 16) + s1[0], u2f(y2 & 0xFFFF0000u) + s1[1]),
                 bf16x2_rne(u2f(y3 << 16) + s1[2], u2f(y3 & 0xFFFF0000u) + s1[3])};
      if ((none >> m) & 1) o = y[i];
      if (((write >> m) & 1) == 0 || t0 + m >= p.T) continue;
      uint16_t* out = p.out + (t0 + m) * p.N + n;
      if constexpr (kWhole) {
        if (there != 0) __builtin_nontemporal_store(o, (u32x4*)out);
      } else if (there == 8) {
        __builtin_memcpy(out, &o, 16);
      } else {
        uint16_t e[8];
        __builtin_memcpy(e, &o, 16);
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (c < there) out[c] = e[c];
      }
    }
  }
};

// The rows (a bit each) that this workgroup writes, of a tile with these adapters: of its own
// adapters, and in the first of a tile's workgroups those without one.
__device__ __forceinline__ uint32_t rows_written(int adapter) {
  bool mine = adapter < 0 && blockIdx.z == 0;
  for_adapters(adapter, [&](int a) { mine = mine || adapter == a; });
  return (uint32_t)__ballot(mine) & 0xFFFFu;
}

// Waves per SIMD that the registers have to be enough for. Left to itself the compiler takes 132 with one
// step, room for three (16384 rows of rank 16 65 us, 49 with four), and 272 with seven, room for one (3000
// rows of rank 104, both products, 46, 39 with two). The others keep what they have so: eight steps of
// weights of their own would spill, and rank 128 takes 98 us instead of 92 with its sums moved.
constexpr int up_waves(int steps) { return steps == 1 ? 4 : steps == 7 ? 2 : 1; }

// `tiles` tiles of 16 rows, one after the other; the adapter's fragments of B stay in registers until
// a tile has another. Above 64 ranks the workgroup's waves share a tile's v in LDS, loaded two tiles ahead:
// each for itself, v's bytes are more than those of y and out together (both products, 16384 rows into
// 4096, rank 128: 221 us, shared 161; 3000 of rank 104 93, 39; rank 64 with 8192 rows 66 either way).
template <int kSteps, bool kHalves, int kWaves, Rows kRows>
__global__ void __launch_bounds__(64 * kWaves, up_waves(kSteps)) lora_up_kernel(LoraProblem p, int tiles) {
  typedef UpRows<kWaves, kRows> Part;
  typedef UpWeights<kSteps, kHalves> Weights;
  constexpr bool kShared = kSteps > 4;
  constexpr int kAll = Weights::kAll, kVChunks = lora_tile_chunks(16 * kSteps);  // (at most)
  constexpr int kVLoads = kShared ? (kVChunks + 64 * kWaves - 1) / (64 * kWaves) : 1;
  __shared__ __align__(16) float sums[2][16 * Part::kPitch];
  __shared__ u32x4 vs[kShared ? 2 : 1][kShared ? kVChunks : 1];
  const int lane = threadIdx.x & 63, q = lane >> 4, r = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t first = (int64_t)blockIdx.x * (64 * kWaves), n0 = first + 64 * wave;
  const int64_t t0 = (int64_t)blockIdx.y * (16 * tiles);
  const int64_t last = (p.T - 1) >> 4;  // tile
  struct Tile {
    u32x4 v[kShared ? 1 : kAll];
    Part rows;
    int adapter;
    uint32_t write;
  };
  auto load = [&](Tile& k, int j) {
    const int64_t t = t0 + 16 * j + r;
    k.adapter = adapter_of(p, t);
    k.write = gridDim.z > 1 ? rows_written(k.adapter) : 0xFFFFu;
    if constexpr (!kShared) {
      const u32x4* v = v_tile(p, min((t0 >> 4) + j, last));
#pragma unroll
      for (int i = 0; i < kAll; ++i) k.v[i] = v_chunk(v, i, kSteps, p.R, q, r);
    }
    k.rows.load(p, t0 + 16 * j, k.write);
  };
  // a thread's part of a tile's v
  u32x4 part[kVLoads];
  auto load_v = [&](int j) {
#pragma unroll
    for (int i = 0; i < kVLoads; ++i) {
      const int at = min(i * 64 * kWaves + (int)threadIdx.x, lora_tile_chunks(p.R) - 1);
      part[i] = v_tile(p, min((t0 >> 4) + j, last))[at];
    }
  };
  auto share_v = [&](int j) {
#pragma unroll
    for (int i = 0; i < kVLoads; ++i) {
      const int at = i * 64 * kWaves + (int)threadIdx.x;
      if (at < lora_tile_chunks(p.R)) vs[j & 1][at] = part[i];
    }
  };
  auto meet = [&]() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
  };
  int held = -1;
  Weights w;
  Tile now{{}, Part(p, first), -1, 0u}, next{{}, Part(p, first), -1, 0u};
  load(now, 0);
  if (tiles == 1 && now.write == 0) return;  // nothing for this one of a tile's workgroups
  if constexpr (kShared) {
    load_v(0);
    share_v(0);
    if (tiles > 1) load_v(1);
    meet();
  }
#pragma unroll 1
  for (int j = 0; j < tiles; ++j) {
    if (j + 1 < tiles) load(next, j + 1);
    if constexpr (kShared) {
      if (j + 1 < tiles) share_v(j + 1);
      if (j + 2 < tiles) load_v(j + 2);
    }
    floatx4 sum[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[i] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    for_adapters(now.adapter, [&](int a) {
      if (a != held) w.load(p, a, n0, q, r);
      held = a;
      if constexpr (kShared) {
        u32x4 v[kAll];
#pragma unroll
        for (int k = 0; k < kAll; ++k) v[k] = v_chunk(vs[j & 1], k, kSteps, p.R, q, r);
        w.multiply(sum, v, now.adapter == a, p.R, q);
      } else {
        w.multiply(sum, now.v, now.adapter == a, p.R, q);
      }
    });
    float* s = sums[j & 1];  // (a buffer is written again behind the next tile's barrier)
    Part::put(s, sum, wave, q, r);
    meet();
    now.rows.store(p, s, t0 + 16 * j, now.write, (uint32_t)__ballot(now.adapter < 0));
    if constexpr (!kShared) {
#pragma unroll
      for (int i = 0; i < kAll; ++i) now.v[i] = next.v[i];
    }
    now.rows.y[0] = next.rows.y[0];
    now.rows.y[1] = next.rows.y[1];
    now.adapter = next.adapter;
    now.write = next.write;
  }
}

// ---- both in one launch, for few rows ----
//
// Every workgroup of 512 columns computes the v that it needs for itself, from the caches: a launch
// less (of 3 us on the host and as much on the device) for as many readings of A.
template <int kR, int kC, int kSteps, bool kHalves, Rows kRows>
__global__ void __launch_bounds__(512) lora_small_kernel(LoraProblem p) {
  constexpr int kWaves = 8, kBytes = kUnitBytes<kR, kC>;
  typedef UpRows<kWaves, kRows> Part;
  typedef UpWeights<kSteps, kHalves> Weights;
  static_assert(kWaves * kBytes >= 64 * Part::kPitch && kBytes >= kR * 1024, "what follows is held in the same memory");
  __shared__ __align__(16) uint8_t lds[kWaves * kBytes];
  __shared__ u32x4 parts[lora_tile_chunks(16 * kR)];
  const int lane = threadIdx.x & 63, q = lane >> 4, r = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t first = (int64_t)blockIdx.x * (64 * kWaves), n0 = first + 64 * wave;
  const int64_t t0 = (int64_t)blockIdx.y * 16;
  const int adapter = adapter_of(p, t0 + r);
  const uint32_t write = rows_written(adapter);
  if (write == 0) return;  // nothing for this one of a tile's workgroups
  Part rows(p, first);
  rows.load(p, t0, write);
  floatx4 sum[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) sum[i] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  const __amdgpu_buffer_rsrc_t rx = x_window(p, t0, 16);
  for_adapters(adapter, [&](int a) {
    Weights w;
    w.load(p, a, n0, q, r);
    const float s = p.scales ? p.scales[a] : 1.0f;
    floatx4 acc[kR];
    down_units<kR, kC, kWaves>(acc, rx, a_window(p, a, 0, 16 * kR), (uint32_t)(p.K * 2), (int)(p.K >> 3), wave, lane,
                               lds + wave * kBytes);
    __syncthreads();
    floatx4* part = (floatx4*)lds;
#pragma unroll
    for (int i = 0; i < kR; ++i) part[(wave * kR + i) * 64 + lane] = acc[i];
    __syncthreads();
    if (wave < kR && 16 * wave + 4 * q < p.R)
      store_parts(parts, r, 16 * wave + 4 * q, p.R, down_sum<kR, kWaves>(part, wave, lane) * s);
    __syncthreads();
    u32x4 v[Weights::kAll];
#pragma unroll
    for (int k = 0; k < Weights::kAll; ++k) v[k] = v_chunk(parts, k, kSteps, p.R, q, r);
    w.multiply(sum, v, adapter == a, p.R, q);
  });
  __syncthreads();
  Part::put((float*)lds, sum, wave, q, r);
  __syncthreads();
  rows.store(p, (const float*)lds, t0, write, (uint32_t)__ballot(adapter < 0));
}

template <int kSteps, bool kHalves>
void launch_up(const LoraProblem& p, const LoraForm& f, hipStream_t stream) {
  constexpr int kWaves = 4;
  const int64_t columns = 64 * kWaves, rows = 16 * f.up_tiles;
  const dim3 grid((unsigned)((p.N + columns - 1) / columns), (unsigned)((p.T + rows - 1) / rows), (unsigned)f.up_deal);
  const dim3 block(64 * kWaves);
  if (p.N % 8 != 0) hipLaunchKernelGGL((lora_up_kernel<kSteps, kHalves, kWaves, Rows::kAny>), grid, block, 0, stream, p, f.up_tiles);
  else if (f.passing) hipLaunchKernelGGL((lora_up_kernel<kSteps, kHalves, kWaves, Rows::kPassing>), grid, block, 0, stream, p, f.up_tiles);
  else hipLaunchKernelGGL((lora_up_kernel<kSteps, kHalves, kWaves, Rows::kWhole>), grid, block, 0, stream, p, f.up_tiles);
}

template <int kR, int kC, int kWaves>
void launch_down(const LoraProblem& p, const LoraForm& f, hipStream_t stream) {
  const dim3 grid((unsigned)((p.T + 15) / 16 * ((p.R + 16 * kR - 1) / (16 * kR))), 1, (unsigned)f.deal);
  hipLaunchKernelGGL((lora_down_kernel<kR, kC, kWaves>), grid, dim3(64 * kWaves), 0, stream, p);
}

template <int kR, int kTok, int kSplit, int kC, int kBufs>
void launch_down_wide(const LoraProblem& p, hipStream_t stream) {
  const dim3 grid((unsigned)((p.T + 16 * kTok - 1) / (16 * kTok) * ((p.R + 16 * kR - 1) / (16 * kR))));
  hipLaunchKernelGGL((lora_down_wide_kernel<kR, kTok, kSplit, kC, kBufs>), grid, dim3(64 * kTok * kSplit), 0, stream, p);
}

template <int kR, int kC, int kSteps, bool kHalves>
void launch_small(const LoraProblem& p, const LoraForm& f, hipStream_t stream) {
  const dim3 grid((unsigned)((p.N + 511) / 512), (unsigned)((p.T + 15) / 16), (unsigned)f.deal);
  if (p.N % 8 == 0) hipLaunchKernelGGL((lora_small_kernel<kR, kC, kSteps, kHalves, Rows::kWhole>), grid, dim3(512), 0, stream, p);
  else hipLaunchKernelGGL((lora_small_kernel<kR, kC, kSteps, kHalves, Rows::kAny>), grid, dim3(512), 0, stream, p);
}

}  // namespace

int64_t lora_down_bytes(int64_t T, int64_t N, int64_t K, int64_t R) {
  return lora_form(T, N, K, R).down == LoraDown::kFused ? 0 : (T + 15) / 16 * lora_tile_chunks((int)R) * 16;
}

hipError_t launch_lora(const LoraProblem& p, hipStream_t stream) {
  if (p.T == 0 || p.N == 0) return hipSuccess;
  const LoraForm f = lora_form(p.T, p.N, p.K, p.R);
  if (f.down == LoraDown::kFused) {
    if (p.R <= 16) launch_small<1, 32, 1, false>(p, f, stream);
    else if (p.R == 24) launch_small<2, 16, 2, false>(p, f, stream);
    else launch_small<2, 16, 2, true>(p, f, stream);
    return hipGetLastError();
  }
  if (f.down == LoraDown::kNarrow) launch_down<1, 16, 8>(p, f, stream);
  else if (f.down == LoraDown::kPair) launch_down<2, 16, 8>(p, f, stream);
  else launch_down_wide<4, 2, 2, 16, 3>(p, stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  switch (lora_steps(p.R) * 2 + lora_halves(p.R)) {
    case 2: launch_up<1, false>(p, f, stream); break;
    case 4: launch_up<2, false>(p, f, stream); break;
    case 5: launch_up<2, true>(p, f, stream); break;
    case 6: launch_up<3, false>(p, f, stream); break;
    case 8: launch_up<4, false>(p, f, stream); break;
    case 9: launch_up<4, true>(p, f, stream); break;
    case 10: launch_up<5, false>(p, f, stream); break;
    case 12: launch_up<6, false>(p, f, stream); break;
    case 13: launch_up<6, true>(p, f, stream); break;
    case 14: launch_up<7, false>(p, f, stream); break;
    case 16: launch_up<8, false>(p, f, stream); break;
    case 17: launch_up<8, true>(p, f, stream); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace nvfp4
