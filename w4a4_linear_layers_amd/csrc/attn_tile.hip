// serq_attn_prefill for bf16 on LDS tiles (gfx950).
//
// One workgroup: eight waves of 32 query rows over the same keys. The rows
// are `pack` query heads of one group (they share keys and values) times 256
// / pack positions, so the diagonal wastes little and short sequences fill
// their tiles. Keys pass in tiles of 64 through four places for K and four for V
// in LDS.
//
// Both products are taken transposed on v_mfma_f32_32x32x16_bf16: S^T = K Q^T
// leaves each lane with 32 scores of one query (column = lane % 32) per tile,
// and those registers, converted in order, are the second operand of O^T =
// V^T P^T: the index that the instruction sums over may be renamed, so lane
// half h = lane / 32 takes as its eight slots of 16 keys those it already
// holds (4 h .. 4 h + 3 and 8 + 4 h .. 8 + 4 h + 3). V^T is read from LDS by
// the transposing reads in the same order. Softmax statistics are one value
// per lane, and scores never leave the registers. Weights are rounded to bf16
// for the product with the values, which the instruction wants alike; their sum
// l is of the unrounded ones (outputs 0.0018 to 0.0024 from the 64-bit ones in
// relative norm, 0.0016 to 0.0017 of it their own rounding to bf16).
//
// 16384 tokens of 32 query and 8 key/value heads of 128: 1.78 to 1.91 ms on
// several cards, 1.15 to 1.24 PFLOP/s of the visible pairs (a large bf16
// product reaches 1.39). The matrix cores are busy 69 % of the cycles; under
// this load the card runs at about 1.7 GHz, so what fewer cycles gain its clock
// gives back in part. A period of two tiles (one of either wave of a SIMD)
// takes 2600 cycles, 2048 of them matrix products; a workgroup's start and end
// another 12000.

#include <type_traits>

#include "attn_common.h"

namespace serq {
namespace {

using namespace attn;

constexpr int kWaves = 8;
constexpr int kKeys = 64;          // keys of a tile
constexpr int kRing = 4;           // tiles of K and of V in LDS (a power of two)

typedef short s16x4 __attribute__((ext_vector_type(4)));

// One 16-byte direct global->LDS load per lane, from sbase + voff (sbase
// wave-uniform), into the wave's 1 KB chunk at `lds_chunk`: lane i lands at
// + 16 i. M0 is written here and declared clobbered. The compiler neither
// counts nor waits for these loads: wait_loads() does. Nor does it order them
// with LDS reads: they write where no wave reads until the next barrier but
// one, and barriers and waits order with them (all are volatile).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma16(const void* sbase, uint32_t voff, uint32_t lds_chunk) {
  asm volatile("s_mov_b32 m0, %2\n\tglobal_load_lds_dwordx4 %0, %1"
               :: "v"(voff), "s"(sbase), "s"(lds_chunk) : "m0");
}
// The same from an address of each lane's own.
__device__ __forceinline__ void dma16(const void* src, uint32_t lds_chunk) {
  asm volatile("s_mov_b32 m0, %1\n\tglobal_load_lds_dwordx4 %0, off" :: "v"(src), "s"(lds_chunk) : "m0");
}
#pragma clang diagnostic pop

// Pointer of another lane.
template <typename T>
__device__ __forceinline__ T* shuffle(T* p, int from) {
  const uint64_t x = reinterpret_cast<uint64_t>(p);
  const uint64_t lo = static_cast<uint32_t>(__shfl(static_cast<int>(x), from, 64));
  const uint64_t hi = static_cast<uint32_t>(__shfl(static_cast<int>(x >> 32), from, 64));
  return reinterpret_cast<T*>(hi << 32 | lo);
}

__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_loads_but() { asm volatile("s_waitcnt vmcnt(%0)" :: "n"(N) : "memory"); }

// LDS accesses of this wave done, then the workgroup's barrier.
__device__ __forceinline__ void barrier() {
  __builtin_amdgcn_s_waitcnt(0xC07F);          // lgkmcnt(0), no vmcnt wait
  asm volatile("s_barrier" ::: "memory");
}

__device__ __forceinline__ f32x16 mfma(u32x4 a, u32x4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                 0);
}

// Value over both lane halves: maximum or sum of a lane and lane ^ 32.
__device__ __forceinline__ float max_halves(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_halves(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// LDS image of a tile: 64 rows of D values. The 16-byte part c of row r lies
// at part c ^ swizzle(r), so that rows read together fall on different banks:
// K by reads of one part of 32 rows, V by transposing reads of 64 bytes of
// four rows.
template <int D>
__device__ __forceinline__ int swizzle_k(int r) { return D == 128 ? r & 15 : (r >> 1) & 7; }
template <int D>
__device__ __forceinline__ int swizzle_v(int r) { return D == 128 ? (r & 3) << 2 : ((r >> 1) & 1) << 2; }

// PREFIX: the prefix part of serq_attn_decode instead. The rows are those of
// all sequences (row R: sequence R / G, head R % G of the group), 256 to a
// workgroup, and all of them see all keys.
template <int D, bool PREFIX>
__global__ __launch_bounds__(64 * kWaves, 2) void attn_tile_kernel(AttnArgs a, PrefillPlan p, int chunk,
                                                                   Parts parts) {
  constexpr int kRow = 2 * D;                    // bytes of a row
  constexpr int kTile = kKeys * kRow;            // bytes of a K or V tile
  constexpr int kRows = 1024 / kRow;             // rows of one wave load
  constexpr int kLoads = kTile / (1024 * kWaves);
  constexpr int C = D / 16, DB = D / 32;
  // K tiles, then V tiles, and half a tile per wave counted with them for Q at
  // the start (in K's last place and V's last two, which are loaded only when Q
  // is in registers) and O at the end.
  __shared__ __align__(1024) uint8_t smem[(2 * kRing + 1) * kTile];
  __shared__ __align__(16) int odd_rows[kRing][kWaves];         // V tiles: whether a wave's rows hold NaN or infinities

  const int lane = threadIdx.x & 63, n = lane & 31, half = lane >> 5;
  const int wave = uniform(threadIdx.x >> 6);
  const int G = a.Hq / a.Hkv;
  bool split = PREFIX;
  int row, head, kvh, len, mine, low, high, end;
  int whole;                                     // keys that all rows of the workgroup see
  bool valid;
  const int32_t* table;
  if constexpr (PREFIX) {
    kvh = blockIdx.x % a.Hkv;
    const int rows = a.B * G, R0 = static_cast<int>(blockIdx.x / a.Hkv) * (32 * kWaves) + 32 * wave;
    valid = R0 + n < rows;
    const int R = valid ? R0 + n : rows - 1;
    row = R / G;
    head = kvh * G + R % G;
    len = mine = low = end = whole = a.prefix_len;
    high = R0 < rows ? len : 0;
    table = a.prefix_table;
  } else {
    const int units = a.Hq / p.pack;
    const int unit = blockIdx.x % units;
    TileAt at;
    if (!find_tile<false>(a, p.tile_pos, blockIdx.x / units, at)) return;
    if (p.splits > 1) {
      const int count = parts_for(a, p, at.total, chunk);
      if (static_cast<int>(blockIdx.y) >= count) return;
      split = count > 1;
    }
    const int nq = at.nq, q0 = at.q0, tile_pos = p.tile_pos, tile = at.tile;
    len = at.len;
    head = unit * p.pack + wave % p.pack;
    kvh = head / G;
    const int pos0 = tile * tile_pos + 32 * (wave / p.pack);
    const int pos = pos0 + n;
    valid = pos < nq;
    row = q0 + (valid ? pos : nq - 1);
    const int shift = len - nq + 1;              // keys that position 0 sees
    const auto sees = [&](int i) { return i + shift < 0 ? 0 : i + shift < len ? i + shift : len; };
    mine = sees(pos), low = sees(pos0), high = pos0 < nq ? sees(pos0 + 31) : 0;
    whole = sees(tile * tile_pos);
    end = sees(tile * tile_pos + tile_pos - 1);  // keys that any row of the workgroup sees
    table = a.page_table + static_cast<int64_t>(at.b) * a.max_pages;
  }
  const int from = static_cast<int>(blockIdx.y) * chunk;
  if (split && end > from + chunk) end = from + chunk;

  u32x4 q[C];              // Q as the second operand: lane (query n, half) holds values 16 c + 8 half .. + 7
  // (Not 0, so that a masked score stays -inf: a scale of 0 becomes the smallest
  // number there is, which makes less than 2^-20 of any product.)
  const float scale = fmaxf(fabsf(a.scale_log2), 0x1p-149f);

  f32x16 o[DB];
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;
  float m = kNone, l = 0.0f;

  const uint32_t lds0 = static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)(&smem[0])));
  const int last = len > 0 ? (len - 1) >> a.page_shift : 0;
  // this lane's share of a wave load: row lane / (kRow / 16) of kRows, one part
  const int lr = lane / (kRow / 16), lp = lane % (kRow / 16);
  uint32_t koff[kLoads], voff[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int r = kRows * (wave + kWaves * i) + lr;
    koff[i] = lr * kRow + ((lp ^ swizzle_k<D>(r)) << 4);
    voff[i] = lr * kRow + ((lp ^ swizzle_v<D>(r)) << 4);
  }
  // Byte offsets of a tile's rows in either cache, for this wave's loads.
  const uint64_t page_bytes = (static_cast<uint64_t>(a.Hkv) << a.page_shift) * kRow;
  const uint32_t head_bytes = (static_cast<uint32_t>(kvh) << a.page_shift) * kRow;
  const uint32_t in_mask = (1u << a.page_shift) - 1;
  const auto look_up = [&](int t, int (&pages)[kLoads]) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int x = (from + t * kKeys + kRows * (wave + kWaves * i)) >> a.page_shift;
      pages[i] = page_entry(table, x < last ? x : last);
    }
  };
  const auto place = [&](const int (&pages)[kLoads], int t, uint64_t (&at)[kLoads]) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      at[i] = static_cast<uint32_t>(in_cache(pages[i], a.n_pages)) * page_bytes +
              (head_bytes + ((from + t * kKeys + kRows * (wave + kWaves * i)) & in_mask) * kRow);
  };
  // V tile t, which some row of the workgroup does not see whole, has landed:
  // this wave's rows past the end, where the cache may hold anything, are
  // cleared, and it is noted whether the others are finite.
  const auto look_over = [&](int t, int slot) {
    bool ok = true;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int r = kRows * (wave + kWaves * i) + lr;
      u32x4* at = reinterpret_cast<u32x4*>(smem + (kRing + slot) * kTile + r * kRow + lp * 16);
      if (from + t * kKeys + r >= len) {
        *at = u32x4{0, 0, 0, 0};
      } else {
        const u32x4 v = *at;
#pragma unroll
        for (int e = 0; e < 4; ++e) ok &= (v[e] & 0x7F80u) != 0x7F80u && (v[e] & 0x7F800000u) != 0x7F800000u;
      }
    }
    const int odd = __any(!ok);
    if (lane == 0) odd_rows[slot][wave] = odd;
  };

  // Read addresses. K: part 2 c + half of row n (+ 32): its swizzled place is
  // that of c = 0 with 2 c flipped in. V: lane i of a group of 16 names 8
  // bytes of row 4 half + i / 4, of the 16 values d % 32 / 16 = lane / 16 % 2.
  const int kbase = n * kRow + ((half ^ swizzle_k<D>(n)) << 4);
  const int vr = 4 * half + ((lane & 15) >> 2);
  const int vpart = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
  const int vbase = kRing * kTile + vr * kRow + ((vpart ^ swizzle_v<D>(vr)) << 4) + 8 * (lane & 1);

  // (The bases of a tile are made opaque: left to itself the compiler keeps all
  // twelve addresses of all stages in registers, and spills them.)
  const auto v_place = [&](int slot) {
    int base = vbase + slot * kTile;
    asm("" : "+v"(base));
    return base;
  };
  const auto v_operand = [&](int base, int d, int j) {
    const uint8_t* at = smem + (base ^ (d << 6)) + 16 * j * kRow;
    typedef __attribute__((address_space(3))) s16x4 lds4;
    const u32x2 x = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(at)));
    const u32x2 y = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(at + 8 * kRow)));
    return u32x4{x[0], x[1], y[0], y[1]};
  };

  f32x16 s[2];                           // scores: register i of block kb is key 32 kb + 8 (i / 4) + 4 half + i % 4
  u32x4 w[4];                            // weights of 16 keys each, in bf16

  const auto scores = [&](int slot) {
    int base = kbase + slot * kTile;
    asm("" : "+v"(base));
#pragma unroll
    for (int i = 0; i < 16; ++i) s[0][i] = s[1][i] = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
        s[kb] = mfma(*reinterpret_cast<const u32x4*>(smem + (base ^ (c << 5)) + 32 * kb * kRow), q[c],
                     s[kb]);
    }
  };

  // Order of a matrix phase: LDS reads kAhead products before their use.
  const auto feed_matrix = [&] {
    constexpr int kAhead = 6, kProducts = 2 * C + 4 * DB;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
#pragma unroll
    for (int i = 0; i < kProducts; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
      if (i + kAhead < 2 * C) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      else if (i + kAhead < kProducts) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
    }
  };

  const auto softmax = [&](int t, auto with_mask) {
    asm volatile("" : "+v"(s[0]), "+v"(s[1]));       // (not before: the compiler would start it among the products)
    if constexpr (decltype(with_mask)::value) {
      const int seen = mine - (from + t * kKeys) - 4 * half;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[kb][i] = 32 * kb + 8 * (i / 4) + (i & 3) < seen ? s[kb][i] : kNone;
    }
    float top = fmaxf(s[0][0], s[1][0]);
#pragma unroll
    for (int i = 1; i < 16; ++i) top = fmaxf(fmaxf(top, s[0][i]), s[1][i]);
    top = max_halves(top) * scale;
    // The exponentials' reference need not be the maximum itself: it follows
    // only where the maximum has outgrown it by 2^8, so that sums and weights
    // are rarely scaled (weights stay below 2^8, their relative rounding the
    // same).
    if (__any(top > m + 8.0f)) {
      const float mn = top > m + 8.0f ? top : m;       // a query's own scores alone decide
      const float f = exp2_(m - ref(mn));
      m = mn;
      l *= f;
#pragma unroll
      for (int d = 0; d < DB; ++d) o[d] *= f;
    }
    const float r = ref(m);
    float sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const float x = exp2_(__builtin_fmaf(s[kb][i], scale, -r));
        const float y = exp2_(__builtin_fmaf(s[kb][i + 1], scale, -r));
        sum[0] += x;
        sum[1] += y;
        w[2 * kb + i / 8][(i / 2) & 3] = pack2(x, y);
      }
    }
    l += sum[0] + sum[1];
    // (done in this phase: left to itself the compiler moves them to the weights' use)
    asm volatile("" : "+v"(w[0]), "+v"(w[1]), "+v"(w[2]), "+v"(w[3]), "+v"(l));
  };

  const auto values = [&](int slot, auto&& between) {
    const int base = v_place(slot);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int d = 0; d < DB; ++d) o[d] = mfma(v_operand(base, d, j), w[j], o[d]);
      between(j);
    }
  };

  // The product of a tile that not all queries see whole. Where one of its
  // values is not finite, 0 * inf would not be 0: each query then takes the
  // product over its own keys with the others' values cleared.
  const auto masked_values = [&](int t, int slot) {
    int odd = 0;
    if (from + (t + 1) * kKeys > whole) {
#pragma unroll
      for (int i = 0; i < kWaves; ++i) odd |= odd_rows[slot][i];
    }
    if (!uniform(odd)) {
      __builtin_amdgcn_sched_barrier(0);
      values(slot, [](int) {});
#pragma unroll
      for (int i = 0; i < 6; ++i) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
#pragma unroll
      for (int i = 0; i < 4 * DB; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
        if (i + 6 < 4 * DB) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
      return;
    }
#pragma unroll
    for (int d = 0; d < DB; ++d) {
      for (int i = 0; i < 32; ++i) {
        const int seen = __shfl(mine, i, 64) - (from + t * kKeys) - 4 * half;
        f32x16 x = o[d];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          u32x4 v = v_operand(v_place(slot), d, j);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int k0 = 16 * j + 8 * (e / 2) + 2 * (e & 1);
            v[e] = (k0 < seen ? v[e] & 0xFFFFu : 0u) | (k0 + 1 < seen ? v[e] & 0xFFFF0000u : 0u);
          }
          x = mfma(v, w[j], x);
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) o[d][e] = n == i ? x[e] : o[d][e];
      }
    }
  };

  // The waves of a SIMD (w and w + 4) work in opposite phases, so that one
  // feeds the matrix cores while the other takes its exponentials. A wave's
  // matrix phase of tile t is S(t) and the product of tile t - 1, its vector
  // phase the softmax of tile t. Period t, with one barrier at its end, is
  // matrix phase t and vector phase t in the first group of four waves, vector
  // phase t - 1 and matrix phase t in the second.
  //
  // In its matrix phase of tile t a wave starts its share of the loads of K(t
  // + kRing - 1) and V(t + kRing - 2), into the places of K(t - 1) and V(t -
  // 2), last read in period t - 1; at the end of period t it waits for K(t +
  // 1) and V(t), while the kRing - 2 batches after them are under way. Every
  // batch has the same number of loads: past the last tile they fetch its pages
  // again, into places no longer read. (Four places: keys that no other
  // workgroup has fetched yet come from HBM.)
  const int steps = from < end ? (end - from + kKeys - 1) / kKeys : 0;
  const bool second = wave >= kWaves / 2;
  if (steps > 0) {
    int pages[kLoads];                             // of the next K tile to load
    uint64_t kat[kLoads], vat[kLoads];             // rows of the K and V tile to load
    int t = 0, slot = 0;                           // tile t and its place
    const auto place_of = [&](int ahead) { return (slot + ahead) & (kRing - 1); };
    const auto load_k = [&](int i, int at) {
      dma16(static_cast<const char*>(a.Kc) + kat[i], koff[i], uniform(lds0 + at * kTile + 1024 * (wave + kWaves * i)));
    };
    const auto load_v = [&](int i, int at) {
      dma16(static_cast<const char*>(a.Vc) + vat[i], voff[i],
            uniform(lds0 + (kRing + at) * kTile + 1024 * (wave + kWaves * i)));
    };
    const auto start_load = [&](int j) {           // of 2 kLoads: V(t + kRing - 2), K(t + kRing - 1)
      if (j < kLoads) {
        load_v(j, place_of(kRing - 2));
      } else if (j < 2 * kLoads) {
        if (j == kLoads) place(pages, t + kRing - 1, kat);
        load_k(j - kLoads, place_of(kRing - 1));
        vat[j - kLoads] = kat[j - kLoads];
      }
    };
    const auto finish_loads = [&] {                // K(t + 1), V(t)
      wait_loads_but<(kRing - 2) * 2 * kLoads>();
      if (from + (t + 1) * kKeys > whole) look_over(t, slot);
    };
    const auto after_matrix = [&](bool ends) {
      if (ends) {
        finish_loads();
        barrier();
      }
      look_up(t + kRing, pages);                   // (a scalar load; among LDS reads it would stall them)
    };
    const auto after_vector = [&](bool ends) {
      if (ends) {
        finish_loads();
        barrier();
      }
      slot = place_of(1);
      ++t;
    };
    int early[kRing - 1][kLoads];
#pragma unroll
    for (int u = 0; u < kRing - 1; ++u) look_up(u, early[u]);
    look_up(kRing - 1, pages);
    // Q by whole rows through LDS: read as an operand from memory, each load
    // would touch 32 rows, 4000 cycles for the workgroup's 64.
    const int qplace = wave < 2 ? (kRing - 1) * kTile + wave * (kTile / 2)
                                : (2 * kRing - 2) * kTile + (wave - 2) * (kTile / 2);
    const char* qrow = reinterpret_cast<const char*>(static_cast<const __bf16*>(a.Q) + row * a.ldq +
                                                     static_cast<int64_t>(head) * D);
#pragma unroll
    for (int k = 0; k < 32 / kRows; ++k) {
      const int r = kRows * k + lr;
      dma16(shuffle(qrow, r) + ((lp ^ swizzle_k<D>(r)) << 4), uniform(lds0 + qplace + 1024 * k));
    }
#pragma unroll
    for (int u = 0; u < kRing - 1; ++u) {          // K(u) and V(u - 1)
      place(early[u], u, kat);
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        load_k(i, u);
        if (u > 0) load_v(i, u - 1);
        vat[i] = kat[i];
      }
    }
    wait_loads_but<(kRing - 2) * 2 * kLoads>();    // Q, K(0)
    // A negative scale goes into Q's sign, so that the largest product is the
    // largest score.
    const uint32_t flip = a.scale_log2 < 0.0f ? 0x80008000u : 0u;
#pragma unroll
    for (int c = 0; c < C; ++c) q[c] = *reinterpret_cast<const u32x4*>(smem + qplace + (kbase ^ (c << 5))) ^ flip;
    barrier();
#pragma unroll
    for (int j = 0; j < 2 * kLoads; ++j) start_load(j);
    scores(slot);
    after_matrix(second);
    // Tiles that all of the wave's queries see whole, then the others. (The
    // waves change over at tiles of their own, and pass the same barriers in
    // either loop.) No whole tile reaches past the end: low <= len.
    const auto whole_tiles = [&](auto second_group) {
      constexpr bool kSecond = decltype(second_group)::value;
      while (t + 1 < steps && from + (t + 1) * kKeys <= low) {
        softmax(t, std::false_type{});
        after_vector(!kSecond);
        __builtin_amdgcn_s_setprio(1);
        __builtin_amdgcn_sched_barrier(0);
        scores(slot);
        values(place_of(kRing - 1), start_load);
        feed_matrix();
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(0);
        after_matrix(kSecond);
      }
    };
    if (second) whole_tiles(std::true_type{});
    else whole_tiles(std::false_type{});
    while (true) {
      if (from + t * kKeys < high) softmax(t, std::true_type{});
      after_vector(!second);
      if (t < steps) {
#pragma unroll
        for (int j = 0; j < 2 * kLoads; ++j) start_load(j);
        if (from + t * kKeys < high) scores(slot);
      }
      if (from + (t - 1) * kKeys < high) masked_values(t - 1, place_of(kRing - 1));
      if (t == steps) break;
      after_matrix(second);
    }
    wait_loads();                                  // nothing may land here after the workgroup is gone
  }

  // o[d][i]: value 32 d + 8 (i / 4) + 4 half + i % 4 of query n. Through LDS,
  // a wave's rows apart, so that rows are stored whole.
  l = sum_halves(l);
  constexpr int kPad = kRow + 16;
  uint8_t* const mine_o = smem + wave * 32 * kPad;
  const auto store_rows = [&](char* to) {          // kRow bytes of each row; `to` of lane r: row r, null for none
    constexpr int N = 32 / kRows;
    char* at[N];
    u32x4 v[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int r = kRows * k + lr;
      at[k] = shuffle(to, r);
      v[k] = *reinterpret_cast<const u32x4*>(mine_o + r * kPad + lp * 16);
    }
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (at[k]) *reinterpret_cast<u32x4*>(at[k] + lp * 16) = v[k];
  };
  barrier();                                       // no wave reads tiles any more
  if (split) {
    // (the join takes only parts that begin before `mine`)
    const bool wanted = valid && (PREFIX || from < mine || from == 0);
    const int64_t slot = (static_cast<int64_t>(row) * a.Hq + head) * parts.splits + blockIdx.y;
    char* to = wanted ? reinterpret_cast<char*>(parts.o + slot * D) : nullptr;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int d = 0; d < DB / 2; ++d) {
        const f32x16& x = o[h * (DB / 2) + d];
#pragma unroll
        for (int i = 0; i < 16; i += 4)
          *reinterpret_cast<f32x4*>(mine_o + n * kPad + (32 * d + 2 * i + 4 * half) * 4) =
              f32x4{x[i], x[i + 1], x[i + 2], x[i + 3]};
      }
      store_rows(to ? to + h * kRow : nullptr);
    }
    if (wanted && half == 0) parts.ml[slot] = float2{m, l};
  } else {
    const float inv = inverse(l);
    if (__any(inv == 0.0f)) {                      // (normed(), apart: few waves have such rows)
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] = inv == 0.0f ? 0.0f : o[d][i];
    }
    char* to = valid ? reinterpret_cast<char*>(static_cast<__bf16*>(a.O) + row * a.ldo + static_cast<int64_t>(head) * D)
                     : nullptr;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<u32x2*>(mine_o + n * kPad + (32 * d + 2 * i + 4 * half) * 2) =
            u32x2{pack2(o[d][i] * inv, o[d][i + 1] * inv), pack2(o[d][i + 2] * inv, o[d][i + 3] * inv)};
    store_rows(to);
  }
}

}  // namespace

hipError_t launch_attn_tile(const AttnArgs& a, const PrefillPlan& p, const Parts& parts, hipStream_t st) {
  const int64_t tiles = static_cast<int64_t>(a.T / p.tile_pos) + a.B;    // at least the sum of the sequences' tiles
  const dim3 grid(static_cast<unsigned>(tiles * (a.Hq / p.pack)), p.splits), block(64 * kWaves);
  if (a.D == 64) attn_tile_kernel<64, false><<<grid, block, 0, st>>>(a, p, 0, parts);
  else attn_tile_kernel<128, false><<<grid, block, 0, st>>>(a, p, 0, parts);
  return hipGetLastError();
}

hipError_t launch_attn_prefix_tile(const AttnArgs& a, int splits, int chunk, const Parts& parts, hipStream_t st) {
  const int64_t rows = static_cast<int64_t>(a.B) * (a.Hq / a.Hkv);
  const int64_t tiles = (rows + 32 * kWaves - 1) / (32 * kWaves);
  const dim3 grid(static_cast<unsigned>(tiles * a.Hkv), splits), block(64 * kWaves);
  if (a.D == 64) attn_tile_kernel<64, true><<<grid, block, 0, st>>>(a, PrefillPlan{}, chunk, parts);
  else attn_tile_kernel<128, true><<<grid, block, 0, st>>>(a, PrefillPlan{}, chunk, parts);
  return hipGetLastError();
}

}  // namespace serq
