// The linear in 8-bit integers for gfx950:
//     Y[m, n] = sx[m] * (sw[n] * sum_k Xq[m, k] Wq[n, k]),
// exact int32 sums on v_mfma_i32_*_i8, whose operands are the bytes as they are
// stored. Three kernels, the operands of two of them by whole lines through LDS:
// few tokens stream the weights from HBM, the workgroup's waves sharing its K;
// more take tiles of 256 x 256, or smaller ones where those would leave compute
// units idle; rows that are no whole 16 bytes take one lane an output.
//
// The matrix instructions take weights as their first operand, so a lane holds
// four consecutive channels of one token at a time, which the epilogue scales
// and stores as one vector.

#include "serq_i8.h"

#include <atomic>
#include <type_traits>
#include <utility>

namespace serq {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

#define SERQ_INLINE __attribute__((always_inline))

constexpr int kKTile = 64;          // bytes of a row in a k-tile
constexpr int kCUs = 256;           // compute units of an MI355X

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 p = {static_cast<__bf16>(lo), static_cast<__bf16>(hi)};
  return __builtin_bit_cast(uint32_t, p);
}

// Outputs of token m, channels n .. n + 3 (those below N).
__device__ __forceinline__ void store4(const I8Args& a, v4i acc, int m, int n, float sx, const float* sw) {
  const int64_t at = static_cast<int64_t>(m) * a.N + n;
  const bool whole = n + 3 < a.N && (a.N & 3) == 0;
  if (a.dbg) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < a.N) a.dbg[at + i] = acc[i];
  }
  float y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = sx * (sw[i] * static_cast<float>(acc[i]));
  if (a.y_bf16) {
    __bf16* out = static_cast<__bf16*>(a.Y) + at;
    if (whole) {
      *reinterpret_cast<u32x2*>(out) = u32x2{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < a.N) out[i] = static_cast<__bf16>(y[i]);
    }
  } else {
    float* out = static_cast<float*>(a.Y) + at;
    if (whole) {
      *reinterpret_cast<f32x4*>(out) = f32x4{y[0], y[1], y[2], y[3]};
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < a.N) out[i] = y[i];
    }
  }
}

__device__ __forceinline__ void load_scales(const I8Args& a, int n, float (&sw)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) sw[i] = a.sw[n + i < a.N ? n + i : a.N - 1];
}

// One 16-byte direct global->LDS load per lane, from sbase + voff (sbase
// wave-uniform), into the wave's 1 KB chunk at `lds_chunk`: lane i lands at
// + 16 i. M0 is written here and declared clobbered. Waits are explicit; LDS
// reads are not ordered with it, as it writes where no wave reads until the
// barrier after the wait for it.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma16(const void* sbase, uint32_t voff, uint32_t lds_chunk) {
  asm volatile("s_mov_b32 m0, %2\n\tglobal_load_lds_dwordx4 %0, %1"
               :: "v"(voff), "s"(sbase), "s"(lds_chunk) : "m0");
}
#pragma clang diagnostic pop

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}

template <int N, typename F, int... I>
__device__ __forceinline__ void static_for_impl(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  static_for_impl<N>(f, std::make_integer_sequence<int, N>{});
}

// ---------------------------------------------------------------- few tokens

// One workgroup: RT tiles of 16 weight rows, all tokens (NT tiles of 16). K
// passes in windows of 512 bytes through STAGES places in LDS, by direct
// global->LDS loads of two rows' 512 bytes each: whole lines, where an operand
// loaded straight into registers takes 64 bytes of each of 16 rows and so half
// of the rate into a compute unit (45 tokens, 14336 x 4096, weights from HBM: 26 us
// against 19, 3.1 TB/s; one of 4096 x 28672 22 us, 5.3 TB/s, a large copy's rate). Wave w
// multiplies bytes 64 w .. of each window, lane (row or token l = lane % 16, g =
// lane / 16) with bytes 16 g of those, by v_mfma_i32_16x16x64_i8; the waves' sums
// meet in LDS.
constexpr int kStreamWaves = 8, kWindow = 64 * kStreamWaves;

template <int RT, int NT, int STAGES, int OCC>
__global__ __launch_bounds__(64 * kStreamWaves, OCC) void i8_stream_kernel(I8Args a) {
  constexpr int CPW = RT + NT, kStage = CPW * 16 * kWindow;       // a window: CPW loads of a wave
  static_assert(CPW * (STAGES - 1) < 64, "vmcnt range");
  static_assert(kStreamWaves * RT * NT * 1024 <= STAGES * kStage, "the sums take the windows' place");
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = blockIdx.x * (16 * RT);
  const uint32_t lds_base = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(lds));
  // Rows of a window: RT * 16 of W, then NT * 16 of X. Load i of wave w: rows 16 i +
  // 2 w and the next. A 16-byte part of a row lies at part ^ (row % 16), so that
  // one part of 16 rows falls on distinct banks.
  const int row = 2 * wave + (lane >> 5), part = (lane & 31) ^ row;
  const int8_t* const wsrc = a.Wq + static_cast<int64_t>(n0) * a.K;
  uint32_t off[CPW];
#pragma unroll
  for (int i = 0; i < CPW; ++i) {
    const int r = 16 * (i < RT ? i : i - RT) + row, last = (i < RT ? a.N - n0 : a.M) - 1;
    off[i] = static_cast<uint32_t>(r < last ? r : last) * a.K + 16 * part;
  }
  const int all = (a.K + kWindow - 1) / kWindow, ragged = a.K % kWindow;
  // (K's ragged end is filled with zeros; part 0 of a row is always there, so
  // every load is issued)
  // Each workgroup of an XCD begins at another window: rows a multiple of 2 KB
  // apart lie in few of its L2's channels, and all workgroups read the tokens.
  const int turn = static_cast<int>(blockIdx.x >> 3) % all;
  const auto issue = [&](int step, int stage) SERQ_INLINE {
    int k = step + turn;
    k -= k >= all ? all : 0;
    const uint32_t to = lds_base + stage * kStage + wave * 1024;
    const bool whole = ragged == 0 || k + 1 < all, in = whole || 16 * part < ragged;
#pragma unroll
    for (int i = 0; i < CPW; ++i) {
      const int8_t* src = (i < RT ? wsrc : a.Xq) + k * kWindow;
      if (whole) dma16(src, off[i], to + i * 8192);
      else if (in) dma16(src, off[i], to + i * 8192);
      else *reinterpret_cast<u32x4*>(lds + stage * kStage + wave * 1024 + i * 8192 + lane * 16) = u32x4{0, 0, 0, 0};
    }
  };
  v4i acc[RT][NT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[r][t] = v4i{0, 0, 0, 0};
  const int at = l * kWindow + (((4 * wave + g) ^ l) << 4);
#pragma unroll
  for (int st = 0; st < STAGES - 1; ++st)
    if (st < all) issue(st, st);
  const auto step = [&](int k, auto sc) SERQ_INLINE {
    constexpr int stage = decltype(sc)::value;
    const int later = all - 1 - k < STAGES - 2 ? all - 1 - k : STAGES - 2;       // windows under way after this one
    static_for<STAGES - 1>([&](auto nc) {
      constexpr int n = decltype(nc)::value;
      if (later == n) wait_vmcnt<CPW * n>();
    });
    __builtin_amdgcn_s_waitcnt(0xC07F);
    asm volatile("s_barrier" ::: "memory");      // window k is there, and nobody reads the one before it any more
    if (k + STAGES - 1 < all) issue(k + STAGES - 1, (stage + STAGES - 1) % STAGES);
    const uint8_t* from = lds + stage * kStage + at;
    v4i w[RT], x[NT];
#pragma unroll
    for (int r = 0; r < RT; ++r) w[r] = *reinterpret_cast<const v4i*>(from + r * 8192);
#pragma unroll
    for (int t = 0; t < NT; ++t) x[t] = *reinterpret_cast<const v4i*>(from + (RT + t) * 8192);
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[r][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[r], x[t], acc[r][t], 0, 0, 0);
  };
  for (int k = 0; k < all; k += STAGES)
    static_for<STAGES>([&](auto sc) {
      if (k + decltype(sc)::value < all) step(k + decltype(sc)::value, sc);
    });
  __builtin_amdgcn_s_waitcnt(0xC07F);
  asm volatile("s_barrier" ::: "memory");
  v4i* red = reinterpret_cast<v4i*>(lds);        // [wave][tile][lane]
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t) red[(wave * RT * NT + r * NT + t) * 64 + lane] = acc[r][t];
  __syncthreads();
  for (int b = wave; b < RT * NT; b += kStreamWaves) {
    v4i sum = red[b * 64 + lane];
#pragma unroll
    for (int i = 1; i < kStreamWaves; ++i) sum += red[(i * RT * NT + b) * 64 + lane];
    const int m = 16 * (b % NT) + l, n = n0 + 16 * (b / NT) + 4 * g;
    if (m < a.M && n < a.N) {
      float sw[4];
      load_scales(a, n, sw);
      store4(a, sum, m, n, a.sx[m], sw);
    }
  }
}

// ---------------------------------------------------------------- tiles

// A 16-byte part of a 64-byte row lies at part ^ swz64(row), so that the reads
// of one part of 16 consecutive rows fall on distinct banks.
__device__ __forceinline__ int swz64(int row) {
  return (((row >> 1) ^ (row >> 2)) & 1) | ((((row >> 2) ^ (row >> 3)) & 1) << 1);
}

// Workgroup -> tile. Workgroups go round-robin over the eight XCDs, each with an
// L2 of its own: each XCD gets a contiguous range of the tile order, which walks
// groups of eight tile rows, a column of a group after another.
__device__ __forceinline__ void tile_coords(int b, int nb, int n_tiles, int& tn, int& tm) {
  constexpr int kXcds = 8, kGroupM = 8;
  const int each = nb / kXcds, more = nb % kXcds, x = b % kXcds;
  const int at = x * each + (x < more ? x : more) + b / kXcds;
  const int m_tiles = nb / n_tiles, per_group = kGroupM * n_tiles;
  const int grp = at / per_group, first = grp * kGroupM;
  const int gm = m_tiles - first < kGroupM ? m_tiles - first : kGroupM;
  const int in = at - grp * per_group;
  tm = first + in % gm;
  tn = in / gm;
}

// One 4-byte direct global->LDS load per lane, likewise: lane i lands at + 4 i.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma4(const void* sbase, uint32_t voff, uint32_t lds_dst) {
  asm volatile("s_mov_b32 m0, %2\n\tglobal_load_lds_dword %0, %1"
               :: "v"(voff), "s"(sbase), "s"(lds_dst) : "m0");
}
#pragma clang diagnostic pop

// The lane's number, found again where it is used: what depends on it alone the
// compiler would otherwise keep over the products, in scratch memory, whose
// loads wait for the tiles' under way.
__device__ __forceinline__ int lane_again() {
  int n;
  asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(n));
  return n;
}

// A tile of 64 TN channels by 64 TM tokens: 2 x 2 waves of TN x TM blocks of 32 x 32
// (v_mfma_i32_32x32x32_i8), over all of K or, with PARTS, one part of it. A
// workgroup takes tiles one after another. (With both ways of storing, 256 x 256
// kept addresses in scratch memory, whose loads wait for those of the next
// tile: 4000 tokens of 4096 x 28672 in 532 us against 460.)
//
// K passes in k-tiles of 64 bytes through STAGES places in LDS, by direct
// global->LDS loads. Lane half h of a block's operands holds bytes 32 h .. + 31
// of its row, the two matrix steps of a k-tile 16 of them each. A wave reads the
// second step's operands during the first step's products and the next
// k-tile's first ones during the second's; between the steps it waits for the
// next k-tile, and after the barrier there nobody reads the present one any
// more, whose place the load of k-tile kt + STAGES takes. The loads stand
// between products: issued at once, they would hold up the products until the
// last is taken.
//
// 4000 tokens, 4096 x 28672: 439 us, 2.14 POPS (the library's 8192^3 product reaches
// 2.06 on this card). Without the outputs' scaling and stores 378 us: the products
// run at 2.5 POPS, near what the loads of 256 x 256 tiles allow (32 KB a k-tile at
// some 32 bytes a clock into a compute unit, the products of a k-tile 1024
// clocks), and the rest is the epilogue, during which the matrix units wait.
// Three places of k-tiles instead of four measure alike (564 us and 558),
// with 128 x 128 up to 6 % more (512 tokens of 8192 x 8192 55 us and 52), with the
// smaller four instead of eight 2 %.
//
// bf16 outputs of 256 x 256 go by whole lines through LDS, 64 channels of a token
// side by side, instead of 32 bytes of a row at a time: 439 us against 460. The
// smaller tiles store as they are (1024 tokens of 8192 x 8192 in 128 x 128: 96 us, 101
// through LDS). fp32 outputs, 16 bytes of a token a lane: 463 us of 4000 tokens against
// 430, 151 of 2048 x 8192 x 8192 against 123; in the smaller tiles within 10 %.
//
// A tile's outputs are stored while the next tile's first k-tiles and its
// scales are under way (the waits count loads, and stores after them make
// them wait for a little more, never for less).
template <int TN, int TM, int STAGES, int OCC, bool PARTS>
__global__ __launch_bounds__(256, OCC) void i8_tile_kernel(I8Args a, int n_tiles, int tiles, int per) {
  constexpr int BN = 64 * TN, BM = 64 * TM;
  constexpr int kW = BN * kKTile, kStage = (BN + BM) * kKTile, CPW = TN + TM;
  constexpr int kScales = STAGES * kStage, kScaleBytes = 4 * (BN + BM);        // two sets of scales after the places,
  constexpr bool kThroughLds = TN == 4 && TM == 4;
  constexpr int kOut = kScales + 2 * kScaleBytes, kOutBytes = 4096;            // then a place of each wave for outputs
  static_assert(CPW * (STAGES - 1) < 64, "vmcnt range");
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  const int lane = threadIdx.x & 63, l32 = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wave >> 1, wm = wave & 1;
  const int all = (a.K + kKTile - 1) / kKTile;
  const int kt0 = static_cast<int>(blockIdx.y) * per;
  const int nkt = all - kt0 < per ? all - kt0 : per;          // k-tiles of this part, at least one
  const int ragged = a.K % kKTile;               // bytes of the last k-tile, 0 for all
  const uint32_t lds_base = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(lds));
  const int part = (lane & 3) ^ swz64(lane >> 2);

  // The tile whose loads are issued: its first rows, and each lane's rows in the
  // wave's chunks of 16 (w TN .. of W, w TM .. of X; rows past the end are the
  // last one again).
  int n0 = 0, m0 = 0;
  const int8_t* wsrc = nullptr;
  const int8_t* xsrc = nullptr;
  uint32_t woff[TN], xoff[TM];
  const auto take = [&](int tile) SERQ_INLINE {
    const int ln = lane_again();
    const int part = (ln & 3) ^ swz64(ln >> 2);
    int tn, tm;
    tile_coords(tile, tiles, n_tiles, tn, tm);
    n0 = __builtin_amdgcn_readfirstlane(tn * BN);
    m0 = __builtin_amdgcn_readfirstlane(tm * BM);
    wsrc = a.Wq + static_cast<int64_t>(n0) * a.K + static_cast<int64_t>(kt0) * kKTile;
    xsrc = a.Xq + static_cast<int64_t>(m0) * a.K + static_cast<int64_t>(kt0) * kKTile;
#pragma unroll
    for (int i = 0; i < TN; ++i) {
      const int row = (wave * TN + i) * 16 + (ln >> 2), last = a.N - 1 - n0;
      woff[i] = static_cast<uint32_t>(row < last ? row : last) * a.K + part * 16;
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int row = (wave * TM + i) * 16 + (ln >> 2), last = a.M - 1 - m0;
      xoff[i] = static_cast<uint32_t>(row < last ? row : last) * a.K + part * 16;
    }
  };
  const auto issue_one = [&](int kt, int stage, int i) SERQ_INLINE {          // chunk i of TN + TM
    const uint32_t to = lds_base + stage * kStage;
    if (i < TN) dma16(wsrc + kt * kKTile, woff[i < TN ? i : 0], to + (wave * TN + i) * 1024);
    else dma16(xsrc + kt * kKTile, xoff[i < TN ? 0 : i - TN], to + kW + (wave * TM + i - TN) * 1024);
  };
  // K's ragged end is filled with zeros. (A load that some lanes skip still
  // counts as one: part 0 of a row is always there.)
  const auto issue = [&](int kt, int stage) SERQ_INLINE {
    if (ragged == 0 || kt0 + kt + 1 < all) {
#pragma unroll
      for (int i = 0; i < TN + TM; ++i) issue_one(kt, stage, i);
      return;
    }
    const uint32_t to = lds_base + stage * kStage;
    const bool in = part * 16 < ragged;
#pragma unroll
    for (int i = 0; i < TN + TM; ++i) {
      const int at = i < TN ? (wave * TN + i) * 1024 : kW + (wave * TM + i - TN) * 1024;
      if (in) dma16(i < TN ? wsrc + kt * kKTile : xsrc + kt * kKTile, i < TN ? woff[i < TN ? i : 0] : xoff[i < TN ? 0 : i - TN], to + at);
      else *reinterpret_cast<u32x4*>(lds + stage * kStage + at + lane * 16) = u32x4{0, 0, 0, 0};
    }
  };
  // The scales of the tile (of channels and tokens that are there) into set
  // `set`, then its first k-tiles.
  const auto begin = [&](int set) SERQ_INLINE {
    const int lane = lane_again();
    const uint32_t to = lds_base + kScales + set * kScaleBytes;
    if (wave == 0) {
#pragma unroll
      for (int c = 0; c < TN; ++c)
        if (n0 + 64 * c + lane < a.N) dma4(a.sw + n0 + 64 * c, 4 * lane, to + 256 * c);
    } else if (wave == 1) {
#pragma unroll
      for (int c = 0; c < TM; ++c)
        if (m0 + 64 * c + lane < a.M) dma4(a.sx + m0 + 64 * c, 4 * lane, to + 4 * BN + 256 * c);
    }
#pragma unroll
    for (int st = 0; st < STAGES; ++st)
      if (st < nkt) issue(st, st);
  };

  v16i acc[TN][TM];
  int wrd[2], xrd[2];
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    wrd[p] = (wn * 32 * TN + l32) * kKTile + (((2 * h + p) ^ swz64(l32)) * 16);
    xrd[p] = kW + (wm * 32 * TM + l32) * kKTile + (((2 * h + p) ^ swz64(l32)) * 16);
  }
  v4i fw[2][TN], fx[2][TM];
  const auto read_one = [&](int stage, auto pc, int i) SERQ_INLINE {           // operand i of TN + TM of a step
    constexpr int p = decltype(pc)::value;
    const uint8_t* sb = lds + stage * kStage;
    if (i < TN) fw[p][i < TN ? i : 0] = *reinterpret_cast<const v4i*>(sb + wrd[p] + i * 32 * kKTile);
    else fx[p][i < TN ? 0 : i - TN] = *reinterpret_cast<const v4i*>(sb + xrd[p] + (i - TN) * 32 * kKTile);
  };
  const auto read_part = [&](int stage, auto pc) SERQ_INLINE {
#pragma unroll
    for (int i = 0; i < TN + TM; ++i) read_one(stage, pc, i);
  };
  // A step's products, with what else is to be issued between them: `with(q)`
  // after product q. The order is kept as it stands here.
  const auto products = [&](auto pc, auto&& with) SERQ_INLINE {
    constexpr int p = decltype(pc)::value;
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j) {
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[p][i], fx[p][j], acc[i][j], 0, 0, 0);
        with(i * TM + j);
        __builtin_amdgcn_sched_barrier(0);
      }
  };
  constexpr int kP = TN * TM, kEvery = kP / (TN + TM) > 0 ? kP / (TN + TM) : 1;      // products to a load
  using P0 = std::integral_constant<int, 0>;
  using P1 = std::integral_constant<int, 1>;
  const auto wait_tiles = [&](int n) SERQ_INLINE {            // until at most n k-tiles are under way
    if (n >= STAGES - 2) {
      wait_vmcnt<CPW * (STAGES - 2)>();
      return;
    }
    static_for<STAGES>([&](auto kc) {
      constexpr int k = decltype(kc)::value;
      if (n == k) wait_vmcnt<CPW * k>();
    });
  };
  const auto step = [&](int kt, int stage, auto whole) SERQ_INLINE {
    constexpr bool kWhole = decltype(whole)::value;          // kt + STAGES is there, and a whole k-tile
    // (a read after each product, the rest after the last)
    const auto reads = [&](int s, auto pc, int q) SERQ_INLINE {
      if (q < TN + TM) read_one(s, pc, q);
      if (q == kP - 1)
#pragma unroll
        for (int i = kP; i < TN + TM; ++i) read_one(s, pc, i);
    };
    __builtin_amdgcn_sched_barrier(0);
    products(P0{}, [&](int q) SERQ_INLINE { reads(stage, P1{}, q); });
    __builtin_amdgcn_s_waitcnt(0xC07F);
    const bool more = kWhole || kt + 1 < nkt;
    if (more) {
      if constexpr (kWhole) wait_vmcnt<CPW * (STAGES - 2)>();
      else wait_tiles(nkt - 2 - kt);
      asm volatile("s_barrier" ::: "memory");
    }
    if constexpr (kWhole) {
      products(P1{}, [&](int q) SERQ_INLINE {
        reads((stage + 1) % STAGES, P0{}, q);
        if (q % kEvery == kEvery - 1 && q / kEvery < TN + TM) issue_one(kt + STAGES, stage, q / kEvery);
        if (q == kP - 1)
#pragma unroll
          for (int i = kP / kEvery; i < TN + TM; ++i) issue_one(kt + STAGES, stage, i);
      });
    } else {
      if (kt + STAGES < nkt) issue(kt + STAGES, stage);
      __builtin_amdgcn_sched_barrier(0);
      if (more) read_part((stage + 1) % STAGES, P0{});
      products(P1{}, [](int) {});
    }
  };

  // Outputs: register e of block (i, j) is channel 32 i + 8 (e / 4) + 4 h + e % 4 of token 32 j + l32.
  const auto four = [&](int i, int j, int q) SERQ_INLINE {
    return v4i{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
  };
  const auto store_parts = [&](int nn, int mm) SERQ_INLINE {
    int32_t* out = a.partial + static_cast<int64_t>(blockIdx.y) * a.M * a.N;
#pragma unroll
    for (int j = 0; j < TM; ++j) {
      const int m = mm + (wm * TM + j) * 32 + l32;
      if (m >= a.M) continue;
#pragma unroll
      for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int n = nn + (wn * TN + i) * 32 + 8 * q + 4 * h;
          int32_t* to = out + static_cast<int64_t>(m) * a.N + n;
          const v4i x = four(i, j, q);
          if (n + 3 < a.N && (a.N & 3) == 0) {
            *reinterpret_cast<v4i*>(to) = x;
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (n + c < a.N) to[c] = x[c];
          }
        }
    }
  };
  const auto store_tile = [&](int nn, int mm, int set) SERQ_INLINE {
    const int ln = lane_again();
    const int l32 = ln & 31, h = ln >> 5;
    const float* ssw = reinterpret_cast<const float*>(lds + kScales + set * kScaleBytes);
    const float* ssx = ssw + BN;
    float sx[TM];
    int m[TM];
#pragma unroll
    for (int j = 0; j < TM; ++j) {
      const int row = (wm * TM + j) * 32 + l32;
      sx[j] = ssx[row];
      m[j] = mm + row;
    }
    const bool pairs = a.y_bf16 && (a.N & 7) == 0 && !a.dbg;
    if (kThroughLds && pairs) {
      // 32 tokens by 64 channels at a time.
      const int r8 = ln >> 3, c8 = ln & 7;
      uint8_t* const mine = lds + kOut + wave * kOutBytes;
      __bf16* const base = static_cast<__bf16*>(a.Y) + static_cast<int64_t>(mm) * a.N + nn;
#pragma unroll
      for (int i = 0; i < TN; i += 2) {
        const int c = (wn * TN + i) * 32 + 8 * c8;
#pragma unroll
        for (int j = 0; j < TM; ++j) {
#pragma unroll
          for (int b = 0; b < 8; b += 2) {                 // blocks of eight channels, two at a time
            uint32_t w[2][2];
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              const int k = i + (b + v) / 4, q = (b + v) % 4;
              const f32x4 sw = *reinterpret_cast<const f32x4*>(ssw + (wn * TN + k) * 32 + 8 * q + 4 * h);
              float y[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) y[e] = sx[j] * (sw[e] * static_cast<float>(acc[k][j][4 * q + e]));
              w[v][0] = pack_bf16x2(y[0], y[1]);
              w[v][1] = pack_bf16x2(y[2], y[3]);
            }
            const auto lo = __builtin_amdgcn_permlane32_swap(w[0][0], w[1][0], false, false);
            const auto hi = __builtin_amdgcn_permlane32_swap(w[0][1], w[1][1], false, false);
            *reinterpret_cast<u32x4*>(mine + l32 * 128 + (((b + h) ^ (l32 & 7)) << 4)) = u32x4{lo[0], hi[0], lo[1], hi[1]};
            asm volatile("" ::: "memory");
          }
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int row = (wm * TM + j) * 32 + 8 * r + r8;
            const u32x4 v = *reinterpret_cast<const u32x4*>(mine + (8 * r + r8) * 128 + ((c8 ^ r8) << 4));
            if (mm + row < a.M && nn + c < a.N) *reinterpret_cast<u32x4*>(base + static_cast<int64_t>(row) * a.N + c) = v;
          }
          asm volatile("" ::: "memory");
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < TN; ++i) {
      const int c0 = (wn * TN + i) * 32;
      f32x4 sw[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) sw[q] = *reinterpret_cast<const f32x4*>(ssw + c0 + 8 * q + 4 * h);
      if (!kThroughLds && pairs) {
        // Lane half h holds channels 8 q + 4 h .. + 3: with the halves of two q
        // exchanged, each lane has eight channels side by side.
#pragma unroll
        for (int j = 0; j < TM; ++j) {
          __bf16* row = static_cast<__bf16*>(a.Y) + static_cast<int64_t>(m[j]) * a.N + nn + c0;
#pragma unroll
          for (int q = 0; q < 4; q += 2) {
            uint32_t w[2][2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              float y[4];
#pragma unroll
              for (int c = 0; c < 4; ++c) y[c] = sx[j] * (sw[q + u][c] * static_cast<float>(acc[i][j][4 * (q + u) + c]));
              w[u][0] = pack_bf16x2(y[0], y[1]);
              w[u][1] = pack_bf16x2(y[2], y[3]);
            }
            const auto lo = __builtin_amdgcn_permlane32_swap(w[0][0], w[1][0], false, false);
            const auto hi = __builtin_amdgcn_permlane32_swap(w[0][1], w[1][1], false, false);
            const int c = 8 * q + 8 * h;
            if (m[j] < a.M && nn + c0 + c < a.N) *reinterpret_cast<u32x4*>(row + c) = u32x4{lo[0], hi[0], lo[1], hi[1]};
          }
        }
        continue;
      }
#pragma unroll
      for (int j = 0; j < TM; ++j) {
        if (m[j] >= a.M) continue;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int n = nn + c0 + 8 * q + 4 * h;
          const float s4[4] = {sw[q][0], sw[q][1], sw[q][2], sw[q][3]};
          if (n < a.N) store4(a, four(i, j, q), m[j], n, sx[j], s4);
        }
      }
    }
  };

  int tile = blockIdx.x, set = 0;
  take(tile);
  begin(set);
  while (true) {
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j) acc[i][j] = v16i{};
    const int later = (nkt < STAGES ? nkt : STAGES) - 1;
    if (later == STAGES - 1) wait_vmcnt<CPW * (STAGES - 1)>();
    else wait_tiles(later);
    __builtin_amdgcn_s_waitcnt(0xC07F);
    asm volatile("s_barrier" ::: "memory");
    read_part(0, P0{});
    int kt = 0;
    for (; kt + 2 * STAGES < nkt; kt += STAGES)
      static_for<STAGES>([&](auto ic) { step(kt + decltype(ic)::value, decltype(ic)::value, std::true_type{}); });
    for (; kt < nkt; kt += STAGES)
      static_for<STAGES>([&](auto ic) {
        constexpr int i = decltype(ic)::value;
        if (kt + i < nkt) step(kt + i, i, std::false_type{});
      });
    const int nn = n0, mm = m0;
    const int now = set;
    tile += gridDim.x;
    const bool more = tile < tiles;
    asm volatile("s_barrier" ::: "memory");      // (every read of the places has landed: its products are issued)
    if (more) {
      take(tile);
      set ^= 1;
      begin(set);
    }
    if constexpr (PARTS) {
      if (a.partial) store_parts(nn, mm);
      else store_tile(nn, mm, now);
    } else {
      store_tile(nn, mm, now);
    }
    if (!more) break;
  }
}

// The parts of K added up, four channels a lane.
__global__ __launch_bounds__(256) void i8_join_kernel(I8Args a, int splits) {
  const int groups = (a.N + 3) / 4;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (at >= static_cast<int64_t>(a.M) * groups) return;
  const int m = static_cast<int>(at / groups), n = static_cast<int>(at % groups) * 4;
  const int64_t part = static_cast<int64_t>(a.M) * a.N;
  const int32_t* from = a.partial + static_cast<int64_t>(m) * a.N + n;
  v4i sum = {0, 0, 0, 0};
  for (int s = 0; s < splits; ++s, from += part) {
    if ((a.N & 3) == 0) {
      sum += *reinterpret_cast<const v4i*>(from);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[i] += n + i < a.N ? from[i] : 0;
    }
  }
  float sw[4];
  load_scales(a, n, sw);
  store4(a, sum, m, n, a.sx[m], sw);
}

// ---------------------------------------------------------------- any K

// (a grid of any size: outputs a lane apart)
__global__ __launch_bounds__(256) void i8_generic_kernel(I8Args a) {
  const int64_t outputs = static_cast<int64_t>(a.M) * a.N, stride = static_cast<int64_t>(gridDim.x) * 256;
  for (int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; at < outputs; at += stride) {
    const int m = static_cast<int>(at / a.N), n = static_cast<int>(at % a.N);
    const int8_t* x = a.Xq + static_cast<int64_t>(m) * a.K;
    const int8_t* w = a.Wq + static_cast<int64_t>(n) * a.K;
    int sum = 0;
    for (int k = 0; k < a.K; ++k) sum += static_cast<int>(x[k]) * w[k];
    if (a.dbg) a.dbg[at] = sum;
    const float y = a.sx[m] * (a.sw[n] * static_cast<float>(sum));
    if (a.y_bf16) static_cast<__bf16*>(a.Y)[at] = static_cast<__bf16>(y);
    else static_cast<float*>(a.Y)[at] = y;
  }
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A kernel's dynamic LDS above 64 KB is allowed once per device (`done`: a bit each).
hipError_t allow_lds(const void* kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (dev < 0 || dev >= 64) return hipErrorInvalidDevice;
  const uint64_t bit = uint64_t{1} << dev;
  if (done.load(std::memory_order_acquire) & bit) return hipSuccess;
  e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess) done.fetch_or(bit, std::memory_order_acq_rel);
  return e;
}

template <int TN, int TM, int STAGES, int OCC, bool PARTS>
hipError_t launch_tile(const I8Args& a, const I8Plan& p, hipStream_t st) {
  constexpr int kLds = 64 * (TN + TM) * (STAGES * kKTile + 8) + (TN == 4 && TM == 4 ? 4 * 4096 : 0);
  const int n_tiles = static_cast<int>(ceil_div(a.N, 64 * TN));
  const int tiles = n_tiles * static_cast<int>(ceil_div(a.M, 64 * TM));
  auto* kernel = &i8_tile_kernel<TN, TM, STAGES, OCC, PARTS>;
  if constexpr (kLds > 64 * 1024) {
    static std::atomic<uint64_t> done{0};
    const hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), kLds, done);
    if (e != hipSuccess) return e;
  }
  const int groups = tiles < OCC * kCUs ? tiles : OCC * kCUs;
  kernel<<<dim3(groups, p.splits), 256, kLds, st>>>(a, n_tiles, tiles, p.per);
  if (p.splits > 1) {
    const int64_t lanes = static_cast<int64_t>(a.M) * ((a.N + 3) / 4);
    i8_join_kernel<<<dim3(static_cast<unsigned>((lanes + 255) / 256)), 256, 0, st>>>(a, p.splits);
  }
  return hipGetLastError();
}

template <int RT, int NT, int STAGES, int OCC>
hipError_t launch_stream(const I8Args& a, hipStream_t st) {
  constexpr int kLds = STAGES * (RT + NT) * 16 * kWindow;
  static_assert(kLds * (OCC / 2) <= 160 * 1024, "LDS");
  auto* kernel = &i8_stream_kernel<RT, NT, STAGES, OCC>;
  if constexpr (kLds > 64 * 1024) {
    static std::atomic<uint64_t> done{0};
    const hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), kLds, done);
    if (e != hipSuccess) return e;
  }
  kernel<<<dim3((a.N + 16 * RT - 1) / (16 * RT)), 64 * kStreamWaves, kLds, st>>>(a);
  return hipGetLastError();
}

// Places: as many as two workgroups a compute unit leave room for, or one
// workgroup where that would be fewer than three.
hipError_t launch_stream_tokens(const I8Args& a, int rt, int nt, hipStream_t st) {
  if (rt == 2) {
    switch (nt) {
      case 1: return launch_stream<2, 1, 3, 4>(a, st);
      case 2: return launch_stream<2, 2, 5, 2>(a, st);
      case 3: return launch_stream<2, 3, 4, 2>(a, st);
      default: return launch_stream<2, 4, 3, 2>(a, st);
    }
  }
  switch (nt) {
    case 1: return launch_stream<1, 1, 5, 4>(a, st);
    case 2: return launch_stream<1, 2, 3, 4>(a, st);
    case 3: return launch_stream<1, 3, 5, 2>(a, st);
    default: return launch_stream<1, 4, 4, 2>(a, st);
  }
}

}  // namespace

I8Plan plan_linear_i8(int M, int K, int N) {
  I8Plan p{};
  p.splits = 1;
  const int k_tiles = static_cast<int>(ceil_div(K, kKTile));
  p.per = k_tiles;
  if (K % 16 != 0) {
    p.kind = I8Kernel::kGeneric;
    p.name = "generic";
    return p;
  }
  if (M <= 64) {
    p.kind = I8Kernel::kStream;
    p.nt = static_cast<int>(ceil_div(M, 16));
    // Weights of two tiles a workgroup, which halves the reads of the tokens, where
    // one tile each would make more workgroups than there are compute units: 45
    // tokens of 4096 x 5120 in 6.9 us against 10.3, 64 of 4096 x 28672 in 36.5 against
    // 47.9; with fewer, 45 of 14336 x 4096 take 22.8 us against 19.3. Few tokens are
    // read quickly either way, and one tile leaves room for twice the workgroups:
    // 16 of 4096 x 32768 in 25.3 us against 28.1, 8 in 25.1 against 25.6, one in 24.7
    // against 24.1; 16 of 4096 x 10240 in 10.4 against 9.9.
    p.rt = p.nt > 2 ? (N > 16 * kCUs ? 2 : 1) : (N >= 16384 && M > 8 ? 2 : 1);
    p.name = "stream";
    return p;
  }
  // Tiles of 256 x 256 take half the loads of 128 x 128 for a product, but go
  // round the 256 compute units one each: two of the smaller side by side take
  // two thirds or more of a large tile's time. 8192 x 8192: 512 tokens 94 us in large
  // tiles and 52 in small ones, 1024 97 and 96, 1280 101 and 122, 2048 126 and 178, 2304
  // 196 and 197, 2900 208 and 244, 4352 309 and 355; 4096 x 28672: 256 tokens 59 and 53,
  // 300 61 and 66, 512 67 and 96, 700 117 and 131; 4096 x 8192: 1024 tokens 49 and 45,
  // 2304 106 and 98, 2900 110 and 123.
  const int64_t tiles = ceil_div(N, 128) * ceil_div(M, 128), big = ceil_div(N, 256) * ceil_div(M, 256);
  if (3 * ceil_div(big, kCUs) <= 2 * ceil_div(tiles, 2 * kCUs)) {
    p.kind = I8Kernel::kTile256;
    p.name = "tile256x256";
    return p;
  }
  // 256 channels by 128 tokens where a unit would have two tiles of 128 x 128 side
  // by side: 1024 tokens of 8192 x 8192 in 87 us against 96, 256 of 4096 x 28672 in 48
  // against 54, 2048 of 14336 x 4096 in 142 against 158, 1000 of 4096 x 6144 in 34
  // against 37; with fewer tiles, 512 of 8192 x 8192 take 75 against 57.
  if (tiles > kCUs) {
    p.kind = I8Kernel::kTile256x128;
    p.name = "tile256x128";
    return p;
  }
  // Tiles of 128 x 128 where there are enough of them; of half that size, or a
  // quarter, where there are not (256 x 4096 x 4096: 11.5 us in tiles of 64 x 64,
  // 17.7 of 128 x 128; 384 tokens 15.1 of 64 x 128, 18.5 of 64 x 64; 768 tokens 21.0 of
  // 128 x 128, 26.6 of 64 x 128). Long rows are cut in parts instead (128 x 14336 x
  // 4096: 25.7 us in eight parts, 29.3 in tiles of 64 x 64 and two; 128 x 8192 x
  // 8192 27.2 in four and 27.5 in tiles of 64 x 64).
  const int64_t quarters = ceil_div(N, 64) * ceil_div(M, 64);
  if (tiles < 150 && k_tiles <= 160) {
    p.kind = quarters <= 256 ? I8Kernel::kTile64 : I8Kernel::kTile64x128;
    p.name = quarters <= 256 ? "tile64x64" : "tile64x128";
    return p;
  }
  p.kind = I8Kernel::kTile128;
  p.name = "tile128x128";
  if (tiles < 150) {
    int64_t s = (256 + tiles / 2) / tiles;
    if (s > k_tiles / 8) s = k_tiles / 8;
    if (s > 16) s = 16;
    if (s > 1) {
      p.per = static_cast<int>(ceil_div(k_tiles, s));
      p.splits = static_cast<int>(ceil_div(k_tiles, p.per));
    }
  }
  if (p.splits > 1) p.bytes = static_cast<int64_t>(p.splits) * M * N * 4;
  return p;
}

hipError_t launch_linear_i8(const I8Args& a, const I8Plan& p, hipStream_t st) {
  switch (p.kind) {
    case I8Kernel::kStream:
      return launch_stream_tokens(a, p.rt, p.nt, st);
    case I8Kernel::kTile256: return launch_tile<4, 4, 4, 1, false>(a, p, st);
    case I8Kernel::kTile256x128: return launch_tile<4, 2, 3, 2, false>(a, p, st);
    case I8Kernel::kTile128: return launch_tile<2, 2, 4, 2, true>(a, p, st);
    case I8Kernel::kTile64x128: return launch_tile<1, 2, 6, 2, false>(a, p, st);
    case I8Kernel::kTile64: return launch_tile<1, 1, 8, 2, false>(a, p, st);
    default: break;
  }
  const int64_t blocks = ceil_div(static_cast<int64_t>(a.M) * a.N, 256);
  i8_generic_kernel<<<dim3(static_cast<unsigned>(blocks < 65536 ? blocks : 65536)), 256, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace serq
