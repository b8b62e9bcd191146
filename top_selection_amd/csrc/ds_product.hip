// Products of 8-bit operands with a scale for each block of 128 along the inner axis.
#include <stddef.h>

#include <type_traits>

#include "ds_expert.h"
#include "ds_rows_device.h"

namespace ds {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));

typedef __bf16 v8h __attribute__((ext_vector_type(8)));
typedef __bf16 v2h __attribute__((ext_vector_type(2)));

// Eight 8-bit floats as bf16, exactly.
template <int ET>
__device__ __forceinline__ v8h widen8(int lo, int hi) {
  v2h p[4];
  if constexpr (ET == DS_E4M3) {
    p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
    p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
    p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  } else {
    p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, 1.0f, false);
    p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, 1.0f, true);
    p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, 1.0f, false);
    p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, 1.0f, true);
  }
  return v8h{p[0][0], p[0][1], p[1][0], p[1][1], p[2][0], p[2][1], p[3][0], p[3][1]};
}

// One block of 128 of sixteen rows of each side: lane l gives 32 of row l % 16's bytes, the same ones on
// both sides (the sum's order is the hardware's), and gets elements (b row 4 (l / 16) + i, a row l % 16).
// As bf16 the products are exact and the sums fp32. The 8-bit unit itself adds eight products at a time, aligned to
// the largest of them, and cuts what is below 2^-13 of it towards zero. Measured against 64 bits (1024 x 1024
// results, k of 128 to 16384 alike), the root mean square of that error over the results' is 1.4e-5 for normal data
// and 3.0e-5 and 5.3e-5 where magnitudes spread over 2^3 and 2^6; where all products have one sign the results are
// short by 2.4e-6, 1.1e-5 and 4.5e-5. A result's rounding to bf16 is 1.7e-3 on that measure.
struct Wide {
  v8h p[4];
};
template <int ET>
__device__ __forceinline__ Wide widen(v8i q) {
  return {widen8<ET>(q[0], q[1]), widen8<ET>(q[2], q[3]), widen8<ET>(q[4], q[5]), widen8<ET>(q[6], q[7])};
}
__device__ __forceinline__ v4f block_product(const Wide& b, const Wide& a) {
  v4f d{0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b.p[i], a.p[i], d, 0, 0, 0);
  return d;
}

// What a workgroup works on.
struct Tile {
  int group;
  int64_t m0, m1;  // rows of a and out
  int64_t k0, k1;  // the inner range
};

__device__ __forceinline__ int64_t clamped(const ProductParams& p, int g, int64_t most) {
  const int64_t v = p.offsets[g];
  return v < 0 ? 0 : v < most ? v : most;
}

// The t-th tile of TM rows of the groups' segments, found by every wave for itself: 64 groups' tiles are
// counted at a time. False past the last.
template <int TM>
__device__ __forceinline__ bool find_rows(const ProductParams& p, int64_t t, Tile& tile) {
  const int lane = threadIdx.x & 63;
  int64_t before = 0;
  for (int g0 = 0; g0 < p.groups; g0 += 64) {
    const int g = g0 + lane;
    int64_t lo = 0, hi = 0;
    if (g < p.groups) {
      lo = clamped(p, g, p.m);
      hi = clamped(p, g + 1, p.m);
    }
    const int tiles = hi > lo ? static_cast<int>((hi - lo + TM - 1) / TM) : 0;
    int incl = tiles;
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(incl, d);
      if (lane >= d) incl += v;
    }
    const uint64_t past = __ballot(t < before + incl);
    if (past) {
      const int at = __ffsll(static_cast<unsigned long long>(past)) - 1;
      const int64_t first = before + __shfl(incl - tiles, at);
      const int slo = __shfl(static_cast<int>(lo), at), shi = __shfl(static_cast<int>(hi), at);
      tile.group = __builtin_amdgcn_readfirstlane(g0 + at);
      tile.m0 = __builtin_amdgcn_readfirstlane(static_cast<int>(slo + (t - first) * TM));
      tile.m1 = __builtin_amdgcn_readfirstlane(shi);
      return true;
    }
    before += __builtin_amdgcn_readlane(incl, 63);
  }
  return false;
}

template <int GROUP, int TM>
__device__ __forceinline__ bool find_tile(const ProductParams& p, int64_t mt, Tile& tile) {
  tile.k0 = 0;
  tile.k1 = p.k;
  if constexpr (GROUP == DS_GROUP_ROWS) return find_rows<TM>(p, mt, tile);
  const int64_t per = (p.m + TM - 1) / TM;
  tile.group = static_cast<int>(mt / per);
  tile.m0 = (mt - tile.group * per) * TM;
  tile.m1 = p.m;
  if constexpr (GROUP == DS_GROUP_INNER) {
    // whole blocks: other offsets count as the next multiple
    const int64_t lo = (clamped(p, tile.group, p.k) + 127) / 128 * 128, hi = (clamped(p, tile.group + 1, p.k) + 127) / 128 * 128;
    tile.k0 = lo < p.k ? lo : p.k;
    tile.k1 = hi < p.k ? hi : p.k;
  }
  return true;
}

// A row's part of a block: 32 bytes a lane, 0 past the end.
__device__ __forceinline__ v8i load_block(const uint8_t* row, int64_t k, int64_t k1, int quad) {
  v4i lo{0, 0, 0, 0}, hi{0, 0, 0, 0};
  const int64_t at = k + quad * 16;
  if (k + 128 <= k1) {  // (the same in all lanes)
    lo = *reinterpret_cast<const v4i*>(row + at);
    hi = *reinterpret_cast<const v4i*>(row + at + 64);
  } else {
    if (at < k1) lo = *reinterpret_cast<const v4i*>(row + at);
    if (at + 64 < k1) hi = *reinterpret_cast<const v4i*>(row + at + 64);
  }
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Few rows: b is read once from memory, straight into registers, and that is what bounds the kernel. A
// workgroup takes 16 MF rows of a and 16 NF of b; its W waves take every W-th block of the inner axis, and their sums
// are joined in LDS in the waves' order. Loads of one block a wave at a time and many waves: with two (four)
// blocks' registers fewer fit (32 rows of 27 experts, 2048 x 4096, 221 MB: 40 us; 42, 52). That is 5.5 TB/s of the
// 6.3 that large reads reach; the rest is finding the segment and the last workgroups' end. The sums
// are exact (block_product): the matrix unit has time.
template <int AT, int BROWS, int GROUP, int OT, int MF, int NF, int W>
__global__ __launch_bounds__(W * 64) void product_small_kernel(ProductParams p) {
  constexpr int TN = NF * 16;
  __shared__ float part[W][64][MF * NF * 4 + 1];
  const int64_t unit = p.unit0 + blockIdx.x;
  Tile t;
  if (!find_tile<GROUP, MF * 16>(p, unit / p.n_tiles, t)) return;
  const int64_t n0 = unit % p.n_tiles * TN;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), row = lane & 15, quad = lane >> 4;
  const int64_t b0 = GROUP == DS_GROUP_ROWS ? t.group * p.n : 0;
  const uint8_t *a[MF], *b[NF];  // (rows past the last repeat it; they are not stored)
  const float *sa[MF], *sb[BROWS == 1 ? NF * 4 : 1];
#pragma unroll
  for (int e = 0; e < MF; ++e) {
    const int64_t m = t.m0 + e * 16 + row < t.m1 ? t.m0 + e * 16 + row : t.m1 - 1;
    a[e] = p.a + m * p.a_stride;
    sa[e] = p.sa + m * p.blocks;
  }
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    const int64_t n = n0 + f * 16 + row < p.n ? n0 + f * 16 + row : p.n - 1;
    b[f] = p.b + (b0 + n) * p.b_stride;
  }
  if constexpr (BROWS == 1) {
#pragma unroll
    for (int q = 0; q < NF * 4; ++q) {
      const int64_t n = n0 + q / 4 * 16 + quad * 4 + q % 4;
      sb[q] = p.sb + (b0 + (n < p.n ? n : p.n - 1)) * p.blocks;
    }
  } else {
    sb[0] = p.sb + ((GROUP == DS_GROUP_ROWS ? t.group * ((p.n + 127) / 128) : 0) + n0 / 128) * p.blocks;
  }
  float acc[MF][NF][4] = {};
  for (int64_t k = t.k0 + wave * 128; k < t.k1; k += W * 128) {
    v8i aq[MF], bq[NF];
    float by_a[MF], by_b[BROWS == 1 ? NF * 4 : 1];
#pragma unroll
    for (int f = 0; f < NF; ++f) bq[f] = load_block(b[f], k, t.k1, quad);
#pragma unroll
    for (int e = 0; e < MF; ++e) {
      aq[e] = load_block(a[e], k, t.k1, quad);
      by_a[e] = sa[e][k / 128];
    }
#pragma unroll
    for (int i = 0; i < (BROWS == 1 ? NF * 4 : 1); ++i) by_b[i] = sb[i][k / 128];
    Wide bw[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) bw[f] = widen<DS_E4M3>(bq[f]);
#pragma unroll
    for (int e = 0; e < MF; ++e) {
      const Wide aw = widen<AT>(aq[e]);
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const v4f sum = block_product(bw[f], aw);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          acc[e][f][i] = __builtin_fmaf(by_a[e] * by_b[BROWS == 1 ? f * 4 + i : 0], sum[i], acc[e][f][i]);
      }
    }
  }
#pragma unroll
  for (int q = 0; q < MF * NF * 4; ++q) part[wave][lane][q] = acc[q / (NF * 4)][q / 4 % NF][q % 4];
  __syncthreads();
  // the fragments' results are shared by the waves
  typename Elem<OT>::T* out = static_cast<typename Elem<OT>::T*>(p.out);
  const int64_t first = GROUP == DS_GROUP_INNER ? t.group * p.m : 0;
  for (int q = wave; q < MF * NF; q += W) {
    float v[4] = {};
#pragma unroll
    for (int w = 0; w < W; ++w)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += part[w][lane][q * 4 + i];
    const int64_t m = t.m0 + q / NF * 16 + row, n = n0 + q % NF * 16 + quad * 4;
    if (m >= t.m1) continue;
    typename Elem<OT>::T* to = out + (first + m) * p.out_stride;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < p.n) to[n + i] = Elem<OT>::narrow(v[i]);
  }
}

// ------------------------------------------------------------------------- tiles through LDS
// The sixteen-byte parts of a tile's rows of 128 lie in LDS in an order that makes a fragment's reads (sixteen
// rows, one part each) meet every bank once, and whose fragments' addresses differ by constants: a's rows
// are consecutive, b's four of each of four runs (Tiled::b_row).
__device__ __forceinline__ int a_part(int row, int part) { return part ^ (row & 7); }
template <int NF>
__device__ __forceinline__ int b_part(int row, int part) {
  return part ^ (((row >> 1) & 1) | (row / (4 * NF) % 4 << 1));
}

// A fragment as the matrix unit takes it: as it is for the 8-bit unit, as bf16 for exact sums.
template <int ET, bool EXACT>
struct Operand {
  v8i v;
  __device__ __forceinline__ void set(v8i q) { v = q; }
};
template <int ET>
struct Operand<ET, true> {
  Wide v;
  __device__ __forceinline__ void set(v8i q) { v = widen<ET>(q); }
};
template <int AT>
__device__ __forceinline__ v4f tile_product(const Operand<DS_E4M3, false>& b, const Operand<AT, false>& a) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b.v, a.v, v4f{0, 0, 0, 0}, 0, AT == DS_E5M2 ? 1 : 0, 0, 0, 0, 0);
}
template <int AT>
__device__ __forceinline__ v4f tile_product(const Operand<DS_E4M3, true>& b, const Operand<AT, true>& a) {
  return block_product(b.v, a.v);
}

// Loads of sixteen (four) bytes a lane from base + offset to LDS from `lds` on, lane after lane, past the
// registers. The compiler holds every LDS read back until such loads have arrived, wherever they write,
// so they are issued behind its back: wait_loads (for all but the newest LEFT) before the barrier that the readers
// wait at.
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const void*)p));
}
// (m0, which says where they go, is declared as written: the compiler warns of any register that it keeps to itself,
// and takes note of the write.)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_to_lds16(const void* base, uint32_t offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(offset), "s"(base), "s"(lds)
               : "m0", "memory");
}
__device__ __forceinline__ void load_to_lds4(const void* base, uint32_t offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1" ::"v"(offset), "s"(base), "s"(lds)
               : "m0", "memory");
}
#pragma clang diagnostic pop
template <int LEFT>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"i"(LEFT) : "memory");
}

// A block of a tile in LDS. Its rows are written and read by sixteen bytes.
template <int TM, int TN, int BROWS>
struct alignas(16) Stage {
  float sa[TM];
  float sb[BROWS == 1 ? TN : 64];
  uint8_t a[TM][128];
  uint8_t b[TN][128];
};

// WM x WN waves, each of MF x NF fragments of sixteen; STAGES blocks in LDS.
//   out = sum over blocks t of sa[., t] sb[., t] d_t, d_t a block's sum from the matrix unit, which starts at 0 for
// every block: its result is scaled and added in vector registers, four multiply-adds for sixteen rows of each side
// (32 cycles of the unit), so that a wave of 128 x 64 has 128 registers of sums and one SIMD two such waves.
// Measured: 8192 x 8192 x 8192 runs at 2.2 PFLOP/s, 64 segments of 1024 +- 300 rows x 4096 x 4096 at 1.77 of live rows
// (1.25 ms; a tenth of the tiles' rows are past their segment). With random operands in registers the unit alone reaches
// 4.0 and with the multiply-adds 3.4 (with zeros 5.0 and 4.2). A block takes 3500 to
// 3700 cycles for the unit's 2048 (2600 without its loads, 3200 with all of them from L2), at the 2.1 GHz that random
// operands leave of 2.4; a tile's start, end and search for its rows are an eighth. Loads of a block sent further ahead
// or spread over its products, four blocks' scales held in registers, tile after tile in one workgroup, other
// orders of tiles, priorities and 32 x 32 fragments all left it there or made it slower.
// For exact sums (EXACT: fp32 results, and bf16 ones that ask for them) the unit takes bf16, of which registers alone
// allow 1.8 PFLOP/s, and 1.5 with the widening (as many vector instructions as the scaling): 8192 x 8192 x 8192 takes
// 950 us (bf16 results 920, where the 8-bit unit takes 500), the segments above 2.08 ms for 1.24, and 16 segments of
// 2048 +- 500 x 4096 x 2048, whose results are 537 MB more, 665 us, 0.82 PFLOP/s.
template <int AT, int BROWS, int GROUP, int OT, bool EXACT, int WM, int WN, int MF, int NF, int STAGES>
struct Tiled {
  static constexpr int kWaves = WM * WN, kThreads = kWaves * 64, TM = WM * MF * 16, TN = WN * NF * 16;
  static constexpr int kLoadsA = TM / 8 / kWaves, kLoadsB = TN / 8 / kWaves;  // of eight rows, a wave
  using S = Stage<TM, TN, BROWS>;
  static constexpr uint32_t kStage = sizeof(S);
  static_assert(alignof(S) == 16 && sizeof(S) % 16 == 0 && offsetof(S, a) % 16 == 0 && offsetof(S, b) % 16 == 0 &&
                offsetof(S, sb) % 16 == 0, "sixteen bytes at a time");

  // A block's rows to LDS: a wave's load is eight rows, its lane l a part of row l / 8.
  // Rows past the last repeat it (they are not stored).
  struct Source {
    const uint8_t* a;
    const uint8_t* b;
    uint32_t ao[kLoadsA], bo[kLoadsB];  // bytes from there
    const float* sa;
    const float* sb;
    uint32_t sao, sbo;
  };

  static __device__ __forceinline__ void stage(S& s, const Source& q, int64_t k, int64_t k1, int wave) {
    if (k + 128 <= k1) {
      const uint8_t* a = q.a + k;
      const uint8_t* b = q.b + k;
#pragma unroll
      for (int i = 0; i < kLoadsA; ++i) load_to_lds16(a, q.ao[i], lds_address(s.a[(i * kWaves + wave) * 8]));
#pragma unroll
      for (int i = 0; i < kLoadsB; ++i) load_to_lds16(b, q.bo[i], lds_address(s.b[(i * kWaves + wave) * 8]));
    } else {
      stage_rest(s, q, k, k1, wave);
    }
    // the scales: a float a row
    const int64_t kb = k / 128;
    if (wave < TM / 64) load_to_lds4(q.sa + kb, q.sao, lds_address(s.sa + wave * 64));
    if constexpr (BROWS == 1) {
      if (wave >= kWaves - TN / 64) load_to_lds4(q.sb + kb, q.sbo, lds_address(s.sb + (wave - (kWaves - TN / 64)) * 64));
    }
  }

  // The last block of an inner length that is no multiple of 128: through registers, zeros past the end.
  static __device__ __forceinline__ void stage_rest(S& s, const Source& q, int64_t k, int64_t k1, int wave) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < kLoadsA + kLoadsB; ++i) {
      const bool of_a = i < kLoadsA;
      const int row = ((of_a ? i : i - kLoadsA) * kWaves + wave) * 8 + lane / 8;
      const int part = of_a ? a_part(row, lane & 7) : b_part<NF>(row, lane & 7);
      uint32_t from = of_a ? q.ao[i % kLoadsA] : q.bo[(i - kLoadsA) % kLoadsB];
      asm volatile("" : "+v"(from));  // (not widened for all of them at once)
      v4i v{0, 0, 0, 0};
      if (k + part * 16 < k1) v = *reinterpret_cast<const v4i*>((of_a ? q.a : q.b) + k + from);
      *reinterpret_cast<v4i*>(of_a ? &s.a[row][(lane & 7) * 16] : &s.b[row][(lane & 7) * 16]) = v;
    }
  }

  // Lane l of a fragment: a row l % 16, and of b the rows whose results make 4 NF consecutive columns a lane.
  static __device__ __forceinline__ int b_row(int f, int lane) {
    return (lane % 16) / 4 * (4 * NF) + f * 4 + lane % 4;
  }

  // Where a lane reads its fragments; it moves from stage to stage.
  struct Places {
    uint32_t sa, sb, a_lo, a_hi, b_lo, b_hi;
    __device__ __forceinline__ void move(uint32_t by) {
      sa += by, sb += by, a_lo += by, a_hi += by, b_lo += by, b_hi += by;
    }
  };
  static __device__ __forceinline__ Places places(const S& s) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, quad = lane >> 4;
    const int m = wave / WN * (MF * 16) + lane % 16, n = wave % WN * (NF * 16), b0 = n + b_row(0, lane);
    return {lds_address(&s.sa[m]),
            lds_address(&s.sb[BROWS == 1 ? n + quad * (4 * NF) : 0]),
            lds_address(&s.a[m][a_part(m, quad) * 16]),
            lds_address(&s.a[m][a_part(m, quad + 4) * 16]),
            lds_address(&s.b[b0][b_part<NF>(b0, quad) * 16]),
            lds_address(&s.b[b0][b_part<NF>(b0, quad + 4) * 16])};
  }
  template <class T>
  static __device__ __forceinline__ T read(uint32_t at) {
    return *reinterpret_cast<const __attribute__((address_space(3))) T*>(at);
  }
  static __device__ __forceinline__ v8i join(uint32_t lo, uint32_t hi) {
    return __builtin_shufflevector(read<v4i>(lo), read<v4i>(hi), 0, 1, 2, 3, 4, 5, 6, 7);
  }

  // What goes from block to block: the fragments (and scales) of b and the first of a, read before the
  // block's products begin, and the last products of the block before, not yet added (a ring of four).
  static constexpr int kLag = 3;
  static_assert(MF * NF % 4 == 0, "the ring starts anew with every block");
  struct State {
    v8i b[NF], a;
    v4f sb[BROWS == 1 ? NF : 1];
    float sa;
    v4f d[4], by[4];
  };
  static __device__ __forceinline__ void read_a(const Places& at, int e, State& h) {
    h.a = join(at.a_lo + e * 2048, at.a_hi + e * 2048);
    h.sa = read<float>(at.sa + e * 64);
  }
  static __device__ __forceinline__ void read_b(const Places& at, int f, State& h) {
    h.b[f] = join(at.b_lo + f * 512, at.b_hi + f * 512);
    if constexpr (BROWS == 1) h.sb[f] = read<v4f>(at.sb + f * 16);
  }
  static __device__ __forceinline__ void add(const State& h, int q, float (&acc)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(h.by[q][BROWS == 1 ? i : 0], h.d[q][i], acc[i]);
    // (without this the compiler moves all of a block's sums behind `turn`, and the products live on)
    asm volatile("" : "+v"(acc[0]), "+v"(acc[1]), "+v"(acc[2]), "+v"(acc[3]));
  }

  // A block of the inner axis. The matrix unit works on the newest products while the one three before is
  // scaled and added and the next fragment of a is read; the order is the source's. When the last fragment of a
  // has been read, `turn` waits for the other waves and moves `at` to the next block's stage, whose fragments
  // replace this one's as their last products are issued.
  template <class F>
  static __device__ __forceinline__ void compute(Places& at, float sb, State& h, float (&acc)[MF][NF][4], F&& turn) {
    Operand<DS_E4M3, EXACT> b[NF];
    Operand<AT, EXACT> a;
#pragma unroll
    for (int e = 0; e < MF; ++e) {
      a.set(h.a);
      const float scale = BROWS == 1 ? h.sa : h.sa * sb;
      if (e == MF - 1) turn();
      read_a(at, (e + 1) % MF, h);
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const int q = e * NF + f, old = (q + MF * NF - kLag) % (MF * NF), now = q % 4;
        if (e == 0) b[f].set(h.b[f]);
        add(h, old % 4, acc[old / NF][old % NF]);
        h.d[now] = tile_product<AT>(b[f], a);
#pragma unroll
        for (int i = 0; i < (BROWS == 1 ? 4 : 1); ++i) h.by[now][i] = BROWS == 1 ? scale * h.sb[f][i] : scale;
        if (e == MF - 1) read_b(at, f, h);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }

  static __device__ __forceinline__ void run(const ProductParams& p, S (&stages)[STAGES]) {
    // eight neighbouring workgroups are on eight XCDs: each XCD takes runs of 32 tiles, whose rows share its L2
    const int64_t id = p.unit0 + blockIdx.x;
    const int64_t unit = (id / 256) * 256 + (id % 8) * 32 + id / 8 % 32;
    if (unit >= p.units) return;
    // tiles in bands of four m tiles, m first
    const int64_t band = 4 * p.n_tiles, of = unit / band, in = unit - of * band;
    const int64_t high = p.m_tiles - of * 4 < 4 ? p.m_tiles - of * 4 : 4;
    Tile t;
    if (!find_tile<GROUP, TM>(p, of * 4 + in % high, t)) return;
    const int64_t n0 = in / high * TN;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t b0 = GROUP == DS_GROUP_ROWS ? t.group * p.n : 0;
    const int mlast = static_cast<int>(t.m1 - t.m0 < TM ? t.m1 - t.m0 : TM) - 1;
    const int nlast = static_cast<int>(p.n - n0 < TN ? p.n - n0 : TN) - 1;
    Source q;
    q.a = p.a + t.m0 * p.a_stride;
    q.b = p.b + (b0 + n0) * p.b_stride;
#pragma unroll
    for (int i = 0; i < kLoadsA; ++i) {
      const int row = (i * kWaves + wave) * 8 + lane / 8;
      q.ao[i] = min(row, mlast) * static_cast<uint32_t>(p.a_stride) + a_part(row, lane & 7) * 16;
    }
#pragma unroll
    for (int i = 0; i < kLoadsB; ++i) {
      const int row = (i * kWaves + wave) * 8 + lane / 8;
      q.bo[i] = min(row, nlast) * static_cast<uint32_t>(p.b_stride) + b_part<NF>(row, lane & 7) * 16;
    }
    q.sa = p.sa + t.m0 * p.blocks;
    q.sao = min(static_cast<int>(threadIdx.x), mlast) * static_cast<uint32_t>(p.blocks) * 4;
    const float* sb_row = p.sb;
    if constexpr (BROWS == 1) {
      q.sb = p.sb + (b0 + n0) * p.blocks;
      q.sbo = min(max(static_cast<int>(threadIdx.x) - (kThreads - TN), 0), nlast) * static_cast<uint32_t>(p.blocks) * 4;
    } else {
      const int64_t b_blocks = (p.n + 127) / 128, at = (n0 + wave % WN * (NF * 16)) / 128;
      sb_row += ((GROUP == DS_GROUP_ROWS ? t.group * b_blocks : 0) + (at < b_blocks ? at : b_blocks - 1)) * p.blocks;
    }
    // The stages in turn: while a block is worked on in one, the next ones are on their way to the others. `turn`:
    // all waves have read block k and the next has arrived; the one that takes block k's place is sent for.
    // (Behind the last block it still waits, and what is read then is not used.)
    int64_t k = t.k0;
    int now = 0;
    const bool extra = wave < TM / 64 || (BROWS == 1 && wave >= kWaves - TN / 64);  // loads scales too
    const auto arrived = [&](auto ahead) {  // all but the loads of the `ahead` newest stages
      constexpr int kLoads = kLoadsA + kLoadsB, kAhead = decltype(ahead)::value;
      static_assert((kLoads + 1) * kAhead < 64, "the counter's range");
      if (k + STAGES * 128 <= t.k1 && kAhead > 0) {
        if (extra) {
          wait_loads<(kLoads + 1) * kAhead>();
        } else {
          wait_loads<kLoads * kAhead>();
        }
      } else {
        wait_loads<0>();  // (near the end fewer stages are under way)
      }
      __syncthreads();
    };
    const auto turn = [&] {
      arrived(std::integral_constant<int, STAGES - 2>{});
      if (k + STAGES * 128 < t.k1) stage(stages[now], q, k + STAGES * 128, t.k1, wave);
      now = now + 1 == STAGES ? 0 : now + 1;
    };
    if (k < t.k1) {
#pragma unroll
      for (int i = 0; i < STAGES; ++i)
        if (k + i * 128 < t.k1) stage(stages[i], q, k + i * 128, t.k1, wave);
      arrived(std::integral_constant<int, STAGES - 1>{});
    }
    if (wave / WN * (MF * 16) > mlast || wave % WN * (NF * 16) > nlast) {
      // the wave's rows or columns lie past the end: it only loads
      for (; k < t.k1; k += 128) turn();
      return;
    }
    float acc[MF][NF][4] = {};
    if (k < t.k1) {
      Places at = places(stages[0]);
      State h{};
      read_a(at, 0, h);
#pragma unroll
      for (int f = 0; f < NF; ++f) read_b(at, f, h);
      float held = 0;  // of 64 blocks a lane holds the scale of one
      for (; k < t.k1; k += 128) {
        float sb = 0;
        if constexpr (BROWS != 1) {
          const int kb = static_cast<int>(k / 128);
          if (kb % 64 == 0) {
            held = sb_row[kb + lane < p.blocks ? kb + lane : p.blocks - 1];
            asm volatile("" : "+v"(held));  // waited for here, and not among the loads to LDS
          }
          sb = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(held), kb % 64));
        }
        compute(at, sb, h, acc, [&] {
          turn();
          at.move(now ? kStage : 0u - (STAGES - 1) * kStage);
        });
      }
#pragma unroll
      for (int q = MF * NF - kLag; q < MF * NF; ++q) add(h, q % 4, acc[q / NF][q % NF]);
    }
    // a lane has 4 NF consecutive columns of MF rows
    const int quad = lane >> 4;
    const int64_t n = n0 + wave % WN * (NF * 16) + quad * (4 * NF);
    typename Elem<OT>::T* out = static_cast<typename Elem<OT>::T*>(p.out);
    const int64_t first = GROUP == DS_GROUP_INNER ? t.group * p.m : 0;
#pragma unroll
    for (int e = 0; e < MF; ++e) {
      const int64_t m = t.m0 + wave / WN * (MF * 16) + e * 16 + lane % 16;
      if (m >= t.m1) continue;
      typename Elem<OT>::T* row = out + (first + m) * p.out_stride;
      if (n + 4 * NF <= p.n) {
        constexpr int V = Elem<OT>::kPer16;
        using Vt = Vec<OT, V>;
#pragma unroll
        for (int c = 0; c < 4 * NF; c += V) {
          typename Vt::type o;
#pragma unroll
          for (int i = 0; i < V; ++i) o[i] = Elem<OT>::narrow(acc[e][(c + i) / 4][(c + i) % 4]);
          *reinterpret_cast<typename Vt::unaligned*>(row + n + c) = o;
        }
      } else {
#pragma unroll
        for (int c = 0; c < 4 * NF; ++c)
          if (n + c < p.n) row[n + c] = Elem<OT>::narrow(acc[e][c / 4][c % 4]);
      }
    }
  }
};

template <int AT, int BROWS, int GROUP, int OT, bool EXACT, int WM, int WN, int MF, int NF, int STAGES>
__global__ __launch_bounds__(WM * WN * 64, 2) void product_tiled_kernel(ProductParams p) {
  using K = Tiled<AT, BROWS, GROUP, OT, EXACT, WM, WN, MF, NF, STAGES>;
  __shared__ typename K::S stages[STAGES];
  K::run(p, stages);
}

// Tiles of TM x TN: how many (an upper bound where the segments decide).
template <int GROUP>
void count_tiles(ProductParams& p, int tm, int tn) {
  p.m_tiles = (p.m + tm - 1) / tm;
  if (GROUP == DS_GROUP_ROWS) p.m_tiles = p.m < p.m / tm + p.groups ? p.m : p.m / tm + p.groups;
  if (GROUP == DS_GROUP_INNER) p.m_tiles *= p.groups;
  p.n_tiles = (p.n + tn - 1) / tn;
  p.units = p.m_tiles * p.n_tiles;
}

template <int AT, int BROWS, int GROUP, int OT, int MF, int NF, int W>
hipError_t small_of(ProductParams& p, hipStream_t s) {
  count_tiles<GROUP>(p, MF * 16, NF * 16);
  return launch_units(product_small_kernel<AT, BROWS, GROUP, OT, MF, NF, W>, p, p.units, W * 64, s);
}

template <int AT, int BROWS, int GROUP, int OT, bool EXACT, int WM, int WN, int MF, int NF, int STAGES>
hipError_t tiled_of(ProductParams& p, hipStream_t s) {
  count_tiles<GROUP>(p, WM * MF * 16, WN * NF * 16);
  return launch_units(product_tiled_kernel<AT, BROWS, GROUP, OT, EXACT, WM, WN, MF, NF, STAGES>, p,
                      (p.units + 255) / 256 * 256, WM * WN * 64, s);
}

// Which kernel. Up to 16 rows (a segment, on average: the host knows no more) b's bytes are all that counts: narrow
// workgroups, the narrower where there are few. Above, the one whose rounds of tiles take least. A round's time
// hardly depends on how full it is; it is a tile's start and end and its blocks of the inner axis (us measured, 8-bit
// unit | exact sums: tiles of 32 x 32 1 + 0.3 a block | 1.5 + 0.45, through LDS 64 x 128 3.5 + 0.5 | 4 + 1, 128 x 128
// 5.6 + 0.7 | 9 + 1.5, 256 x 256 11 + 1.6, and 8 + 1.3 where no tile has more than 128 rows and half of its waves
// only load), and 2 where a segment has to be found (64 x 128: 4). Where tiles share a CU (the smallest; the largest
// of exact sums, two of which hide each other's starts and ends: 665 us for a weights' gradient that 256 x 128 alone
// took 740 for) parts of rounds count. Measured with every kernel forced, bf16 results (32 x 32, 64 x 128, 128 x 128,
// 256 x 256; the chosen one marked):
//   64 segments of 64 rows x 2048 x 4096   311   146*  144   151     128 x 4096 x 4096    22    18*   25    38
//   64 segments of 128 rows, the same      605   202   171   164*    512 x 4096 x 4096    76    19*   27    61
//   64 segments of 300 rows, the same     1418   413   336   257*    1024 x 4096 x 4096  149    36    29*   64
//   64 segments of 100 rows x 2048 x 512   131    49    37    26*    2048 x 4096 x 4096  293    68    53*   65
// The formulas leave out b's bytes, which bound short segments (the first line: 95 us at the least, and 403, 94, 120
// and 103 by formula); what they choose was within 2 % of the best at 24 sizes, with exact sums within 5 % at 17. The
// average misleads where loads are uneven: 64 segments of 16 rows x 2048 x 4096 take 131 us by few rows' kernel and
// 134 by 64 x 128, of 8 rows 114 and 136, but 1024 rows in one of them 110 and 26, 512 rows beside 64 times 8 158 and
// 126.
template <int AT, int BROWS, int GROUP, int OT, bool EXACT>
hipError_t product_of(ProductParams p, hipStream_t s) {
  const int64_t rows = GROUP == DS_GROUP_ROWS ? (p.m + p.groups - 1) / p.groups : p.m;
  const int64_t segments = GROUP == DS_GROUP_NONE ? 1 : p.groups;
  const auto tiles = [&](int tm, int tn) { return segments * ((rows + tm - 1) / tm) * ((p.n + tn - 1) / tn); };
  const auto rounds = [&](int tm, int tn) { return static_cast<double>((tiles(tm, tn) + kCus - 1) / kCus); };
  if (rows <= 16) {
    if (tiles(16, 32) >= 2 * kCus) return small_of<AT, BROWS, GROUP, OT, 1, 2, 8>(p, s);
    return small_of<AT, BROWS, GROUP, OT, 1, 1, 8>(p, s);
  }
  const auto shared = [&](int64_t tiles_, double by) { return tiles_ > kCus / by ? by * tiles_ / kCus : 1.0; };
  const double blocks = static_cast<double>(p.blocks) / (GROUP == DS_GROUP_INNER ? segments : 1);
  const double find = GROUP == DS_GROUP_ROWS ? 2 : 0;
  const auto round = [&](double ends, double block) { return find + ends + block * blocks; };
  const double small = (EXACT ? round(1.5, 0.45) : round(1, 0.3)) * shared(tiles(32, 32), 1.0);
  const double t64 = (find + (EXACT ? round(4, 1) : round(3.5, 0.5))) * rounds(64, 128);
  const double t128 =
      EXACT ? round(9, 1.5) * shared(tiles(128, 128), 0.7) : round(5.6, 0.7) * rounds(128, 128);
  const double t256 = EXACT ? t128 : (rows <= 128 ? round(8, 1.3) : round(11, 1.6)) * rounds(256, 256);
  // (a tile's rows are reached by 32-bit offsets)
  const bool near = p.a_stride < (1 << 23) && p.b_stride < (1 << 23);
  if (!near || (small <= t64 && small <= t128 && small <= t256)) return small_of<AT, BROWS, GROUP, OT, 2, 2, 8>(p, s);
  if (t64 <= t128 && t64 <= t256) return tiled_of<AT, BROWS, GROUP, OT, EXACT, 2, 4, 2, 2, 6>(p, s);
  if constexpr (EXACT) {
    return tiled_of<AT, BROWS, GROUP, OT, EXACT, 2, 2, 4, 4, 2>(p, s);
  } else {
    if (t128 <= t256) return tiled_of<AT, BROWS, GROUP, OT, EXACT, 4, 2, 2, 4, 4>(p, s);
    return tiled_of<AT, BROWS, GROUP, OT, EXACT, 2, 4, 8, 4, 2>(p, s);
  }
}

template <int AT, int OT, bool EXACT>
hipError_t product_by_group(int b_rows, int group, const ProductParams& p, hipStream_t s) {
  if (group == DS_GROUP_INNER) return product_of<AT, 1, DS_GROUP_INNER, OT, EXACT>(p, s);
  if (group == DS_GROUP_ROWS)
    return b_rows == 1 ? product_of<AT, 1, DS_GROUP_ROWS, OT, EXACT>(p, s)
                       : product_of<AT, 128, DS_GROUP_ROWS, OT, EXACT>(p, s);
  return b_rows == 1 ? product_of<AT, 1, DS_GROUP_NONE, OT, EXACT>(p, s)
                     : product_of<AT, 128, DS_GROUP_NONE, OT, EXACT>(p, s);
}

template <int AT>
hipError_t product_by_sums(int b_rows, int group, int out_dtype, bool exact, const ProductParams& p, hipStream_t s) {
  if (out_dtype == DS_FP32) return product_by_group<AT, DS_FP32, true>(b_rows, group, p, s);
  return exact ? product_by_group<AT, DS_BF16, true>(b_rows, group, p, s)
               : product_by_group<AT, DS_BF16, false>(b_rows, group, p, s);
}

}  // namespace

hipError_t launch_product(int a_dtype, int b_rows, int group, int out_dtype, bool exact, ProductParams p, hipStream_t s) {
  return a_dtype == DS_E4M3 ? product_by_sums<DS_E4M3>(b_rows, group, out_dtype, exact, p, s)
                            : product_by_sums<DS_E5M2>(b_rows, group, out_dtype, exact, p, s);
}

}  // namespace ds
