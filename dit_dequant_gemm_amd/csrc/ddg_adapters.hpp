// Low-rank adapters of many requests beside one shared product: row i of Y
// also gets s_a T_i U_a^T with a = rows[i] and T_i = X_i D_a^T.
//
//   adapter_down_kernel   T (times s_a): for at most 64 rows float32 sums over
//                         `chunks` parts of K, which the product adds up in
//                         order; for more rows the bf16 parts of T
//   adapter_tile, adapter_mixed
//                         the branch of a 256-row tile
//   AdapterStage, adapter_first, adapter_rows16
//                         the branch of at most 64 rows
//
// A block of rows may mix adapters.  Every wave walks the distinct adapters of
// its rows (ballots over the ids held one row per lane, so the walk is uniform
// over the wave) and runs the matrix instructions of one adapter at a time,
// the other rows' T as zeros.  Requests are runs of rows, so most blocks hold
// one adapter and cost what one shared adapter does.  An infinity or NaN in
// an adapter's U times another row's zero would be a NaN: mixed tiles take it
// out of the operand and make the outputs of the adapter's own rows infinite,
// mixed blocks of few rows keep an adapter's sums apart and add them to its
// own rows only.
//
// T enters the bf16 matrix instructions as a sum of bf16 parts: two (to 2^-16
// of T) for a bf16 Y, whose own rounding is 2^-8, and three (to 2^-24) for a
// float32 Y.  The products of bf16 values are exact in the float32
// accumulator, so Y is rounded once.
#pragma once

#include "ddg_device.hpp"

namespace ddg {

struct AdapterArgs {
  const int* rows;          // M adapter numbers; outside [0, count): no adapter
  const float* t;           // at most 64 rows: chunks x M x R
  const __bf16* t16;        // more rows: parts x M x R
  const __bf16* up;         // count x N x R
  int count;
  int chunks;
  int parts;
};
struct NoAdapters {};       // a product without them

constexpr int kAdapterMaxChunks = 8;
constexpr int kAdapterMaxParts = 3;

// Row r's adapter, -1 for none and for rows past m.
__device__ __forceinline__ int adapter_of(const int* rows, int count, int r, int m) {
  const int id = rows[min(r, m - 1)];
  return r < m && (unsigned)id < (unsigned)count ? id : -1;
}

// The next bf16 part of t (nearest), which is taken off t.
__device__ __forceinline__ u32x4 take_part(float (&t)[8]) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = pack_bf16x2(t[2 * i], t[2 * i + 1]);
    t[2 * i] -= bf16_bits_to_f32(w[i] & 0xFFFFu);
    t[2 * i + 1] -= __builtin_bit_cast(float, w[i] & 0xFFFF0000u);
  }
  return w;
}

__device__ __forceinline__ bf16x8 keep_or_zero(bf16x8 v, bool keep) {
  return __builtin_bit_cast(bf16x8, keep ? __builtin_bit_cast(u32x4, v) : u32x4{0u, 0u, 0u, 0u});
}

// Any infinity or NaN among the lane's values.
__device__ __forceinline__ bool nonfinite(bf16x8 v) {
  const u32x4 w = __builtin_bit_cast(u32x4, v);
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) bad |= (w[i] & 0x7F80u) == 0x7F80u || (w[i] & 0x7F800000u) == 0x7F800000u;
  return bad;
}

__device__ __forceinline__ f32x16 adapter_mfma(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 adapter_mfma(bf16x8 a, bf16x8 b, f32x4 c) { return mfma16x16x32(a, b, c); }

// An infinity in accumulator c for the rows `mine` in the columns whose U is
// broken (lanes, any k part): the largest bf16 squared; zeros elsewhere.
template <int ROWS, typename Acc>
__device__ __forceinline__ Acc adapter_blow(uint64_t broken, bool mine, Acc c) {
  const bf16x8 big = __builtin_bit_cast(bf16x8, u32x4{0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu});
  const int l = threadIdx.x & (ROWS - 1);
  bool mark = false;
#pragma unroll
  for (int i = 0; i < 64 / ROWS; ++i) mark |= (broken >> (l + i * ROWS)) & 1;
  return adapter_mfma(keep_or_zero(big, mine), keep_or_zero(big, mark), c);
}

// Distinct adapters of up to 64 W rows (id[j]: row 64 j + lane), one at a time.
template <int W>
struct AdapterWalk {
  uint64_t pending[W], match[W];
  int adapter;
  __device__ __forceinline__ explicit AdapterWalk(const int (&id)[W]) {
#pragma unroll
    for (int j = 0; j < W; ++j) pending[j] = __ballot(id[j] >= 0);
  }
  __device__ __forceinline__ bool more() const {
    uint64_t any = 0;
#pragma unroll
    for (int j = 0; j < W; ++j) any |= pending[j];
    return any != 0;
  }
  __device__ __forceinline__ bool next(const int (&id)[W]) {
    bool found = false;
#pragma unroll
    for (int j = 0; j < W; ++j) {
      if (!found && pending[j] != 0) {
        adapter = __builtin_amdgcn_readlane(id[j], __builtin_ctzll(pending[j]));
        found = true;
      }
    }
    if (!found) return false;
#pragma unroll
    for (int j = 0; j < W; ++j) {
      match[j] = __ballot(id[j] == adapter);
      pending[j] &= ~match[j];
    }
    return true;
  }
};

// ---------------------------------------------------------------------------
// 256-row tiles: the branch goes into the accumulators before the K loop.  A
// tile of one adapter (adapter_tile) is straight-line code behind the first
// group's loads, where its latencies overlap theirs.  A tile that mixes
// adapters (adapter_mixed) is done ahead of those loads, while the LDS is
// free: a loop over adapters behind them made the compiler spill around the K
// loop and cost every tile 10 us, also without any adapter.  The branch's
// matrix work is 1 to 2% of the product's; with its latencies and the pre-pass
// it costs 4% at 4096 x 13824 x 5120 and rank 16 (550 us alone, 571 with one
// adapter or requests in runs) and 6% at 32760 x 15360 x 5120 and rank 32 (4.04
// and 4.28 ms, 1.2 PFLOP/s).
//
// ROWS x (256 / ROWS) row blocks, CB column blocks of ROWS from column col0
// on; lane (row or column l, k part q) of the operands.
// ---------------------------------------------------------------------------
template <int ROWS>
struct TileLanes {
  static constexpr int KS = ROWS == 32 ? 16 : 32;             // rank of a matrix instruction
  int l, q;
  __device__ __forceinline__ TileLanes() {
    const int lane = threadIdx.x & 63;
    l = lane & (ROWS - 1);
    q = lane / ROWS;
  }
  // rows `bits` of a row block, for every k part's lanes
  static __device__ __forceinline__ bool mine(uint32_t bits) {
    return __builtin_amdgcn_inverse_ballot_w64(ROWS == 32 ? bits * 0x100000001ull : (bits & 0xFFFFu) * 0x1000100010001ull);
  }
};

// Largest rank of adapter_tile.
constexpr int kAdapterStraight = 32;

template <int ROWS, int CB, typename Acc>
__device__ __forceinline__ void adapter_tile(const AdapterArgs& ad, int m, int n_total, int R, int m0, int col0,
                                             Acc (&acc)[256 / ROWS][CB]) {
  constexpr int RB = 256 / ROWS, KS = TileLanes<ROWS>::KS;
  constexpr int BATCH = 8;                                     // T operands in flight
  const TileLanes<ROWS> tl;
  int id[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) id[j] = adapter_of(ad.rows, ad.count, m0 + 64 * j + (threadIdx.x & 63), m);
  AdapterWalk<4> walk(id);
  if (!walk.next(id) || walk.more() || R > kAdapterStraight) return;
  // T and U through buffer resources: one offset register instead of a 64-bit
  // address per row block; rows past M and columns past N read as zeros
  const uint32_t row_bytes = (uint32_t)R * 2;
  const uint32_t t_bytes = (uint32_t)min(256, m - m0) * row_bytes;
  const uint32_t u_bytes = (uint32_t)max(0, min(CB * ROWS, n_total - col0)) * row_bytes;
  const rsrc_t ru = make_rsrc(ad.up + ((int64_t)walk.adapter * n_total + col0) * R, u_bytes);
  // rows without an adapter: their T was not written, and U may hold
  // infinities, whose product with zero is a NaN
  const bool whole = (walk.match[0] & walk.match[1] & walk.match[2] & walk.match[3]) == ~0ull;
  uint64_t broken[CB] = {};                                    // lanes whose U holds an infinity or a NaN
  auto mine = [&](int rb) { return tl.mine((uint32_t)(walk.match[rb * ROWS / 64] >> (rb * ROWS % 64))); };
  for (int j0 = 0; j0 < R; j0 += KS) {
    const int kk = j0 + 8 * tl.q;
    // a k part past the rank: past the resource, zeros
    const uint32_t off = kk < R ? (uint32_t)tl.l * row_bytes + (uint32_t)kk * 2 : 0x80000000u;
    bf16x8 b[CB];
#pragma unroll
    for (int c = 0; c < CB; ++c) {
      b[c] = __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(ru, off + c * ROWS * row_bytes, 0, 0));
      if (!whole) {
        const bool bad = nonfinite(b[c]);
        broken[c] |= __ballot(bad);
        b[c] = keep_or_zero(b[c], !bad);
      }
    }
    for (int p = 0; p < ad.parts; ++p) {
      const rsrc_t rt = make_rsrc(ad.t16 + ((int64_t)p * m + m0) * R, t_bytes);
#pragma unroll
      for (int r0 = 0; r0 < RB; r0 += BATCH) {
        bf16x8 a[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i)
          a[i] = __builtin_bit_cast(
              bf16x8, __builtin_amdgcn_raw_buffer_load_b128(rt, off + (r0 + i) * ROWS * row_bytes, 0, 0));
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
          a[i] = keep_or_zero(a[i], mine(r0 + i));
#pragma unroll
          for (int c = 0; c < CB; ++c) acc[r0 + i][c] = adapter_mfma(a[i], b[c], acc[r0 + i][c]);
        }
      }
    }
  }
#pragma unroll
  for (int c = 0; c < CB; ++c)
    if (broken[c] != 0) {
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) acc[rb][c] = adapter_blow<ROWS>(broken[c], mine(rb), acc[rb][c]);
    }
}

// A tile of several adapters, or of one whose rank would make adapter_tile a
// chain of load latencies (1517 x 496 x 2560, rank 128: 94 us there, 64 here),
// by the whole workgroup.  T comes through
// LDS, 64 ranks at a time (every adapter's turn reads it again), and so does
// the list of the tile's adapters with their row masks, which the first wave
// writes.  With both at hand the (adapter, rank step) pairs are one sequence:
// U's loads of the next pairs are in flight while one is multiplied, and row
// blocks without the adapter's rows are skipped.  Of the sequence, pairs
// share, share + shares, ... (workgroups that split K share out the pairs
// too).  On return no wave needs the LDS.  A pair over a whole tile takes 1.3
// us, half of it matrix instructions (4096 x 5120 x 5120, 256 adapters in
// every tile: 880 us, 241 with one).
constexpr int kAdapterDepth = 4;                               // pairs whose U is in flight
constexpr int kAdapterFill = 64;                               // ranks of T in LDS
constexpr int kAdapterListAt = kAdapterMaxParts * 256 * kAdapterFill * 2;
constexpr int kAdapterEntry = 5;                               // 64-bit words: row masks, adapter

template <int ROWS, int CB, typename Acc>
__device__ __forceinline__ void adapter_mixed(const AdapterArgs& ad, int m, int n_total, int R, int m0, int col0,
                                              Acc (&acc)[256 / ROWS][CB], uint8_t* lds, int share = 0,
                                              int shares = 1) {
  constexpr int RB = 256 / ROWS, KS = TileLanes<ROWS>::KS;
  constexpr int N = ROWS == 32 ? 512 : 256;                    // lanes of the workgroup
  constexpr int PIECES = KS / 8;                               // 16-byte pieces of a row's rank step
  constexpr int PER = 256 * PIECES / N;                        // pieces per lane, step and part
  constexpr int STEPS = kAdapterFill / KS;
  const TileLanes<ROWS> tl;
  const int tid = threadIdx.x;
  int id[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) id[j] = adapter_of(ad.rows, ad.count, m0 + 64 * j + (tid & 63), m);
  AdapterWalk<4> walk(id);
  // the same in every wave
  if (!walk.next(id) || (!walk.more() && R <= kAdapterStraight)) return;
  uint64_t* list = reinterpret_cast<uint64_t*>(lds + kAdapterListAt);
  if (tid < 64) {
    int count = 0;
    do {
      if (tid == 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) list[1 + count * kAdapterEntry + j] = walk.match[j];
        list[1 + count * kAdapterEntry + 4] = (uint64_t)walk.adapter;
      }
      ++count;
    } while (walk.next(id));
    if (tid == 0) list[0] = (uint64_t)count;
  }
  const uint32_t row_bytes = (uint32_t)R * 2;
  const uint32_t u_bytes = (uint32_t)max(0, min(CB * ROWS, n_total - col0)) * row_bytes;
  for (int f0 = 0; f0 < R; f0 += kAdapterFill) {
    const int steps = (min(R - f0, kAdapterFill) + KS - 1) / KS;
    // T of these ranks: [step][part][row][KS], zeros past the rank and past M
    bf16x8 v[STEPS][kAdapterMaxParts][PER];
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int p = 0; p < kAdapterMaxParts; ++p)
#pragma unroll
        for (int e = 0; e < PER; ++e) {
          const int i = tid + e * N, kk = f0 + s * KS + 8 * (i % PIECES), row = m0 + i / PIECES;
          if (s < steps && p < ad.parts)
            v[s][p][e] = *reinterpret_cast<const bf16x8*>(ad.t16 + ((int64_t)p * m + min(row, m - 1)) * R + min(kk, R - 8));
        }
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int p = 0; p < kAdapterMaxParts; ++p)
#pragma unroll
        for (int e = 0; e < PER; ++e) {
          const int i = tid + e * N, kk = f0 + s * KS + 8 * (i % PIECES), row = m0 + i / PIECES;
          if (s < steps && p < ad.parts)
            *reinterpret_cast<bf16x8*>(lds + ((s * ad.parts + p) * 256 * PIECES + i) * 16) =
                keep_or_zero(v[s][p][e], kk < R && row < m);
        }
    __syncthreads();
    const int count = __builtin_amdgcn_readfirstlane((int)list[0]);
    // the pair (entry of the list, step) to load next and the one to multiply
    int ahead = share / steps, ahead_s = share % steps, at = ahead, s = ahead_s;
    auto advance = [&](int& entry, int& step) __attribute__((always_inline)) {
      step += shares;
      while (step >= steps) {
        step -= steps;
        ++entry;
      }
    };
    bf16x8 b[kAdapterDepth][CB];
    // what the list says of the pair to load next and of the one to multiply
    // next, read a pair early; past the last entry: the last again, not used
    uint32_t ahead_adapter, words[8];
    auto read_ahead = [&]() __attribute__((always_inline)) {
      ahead_adapter = (uint32_t)list[1 + min(ahead, count - 1) * kAdapterEntry + 4];
    };
    auto read_words = [&]() __attribute__((always_inline)) {
      const uint32_t* from = reinterpret_cast<const uint32_t*>(list + 1 + min(at, count - 1) * kAdapterEntry);
#pragma unroll
      for (int i = 0; i < 8; ++i) words[i] = from[i];
    };
    read_ahead();
    read_words();
    auto load_u = [&](bf16x8 (&u)[CB]) __attribute__((always_inline)) {
      const int adapter = __builtin_amdgcn_readfirstlane((int)ahead_adapter);
      const rsrc_t ru = make_rsrc(ad.up + ((int64_t)adapter * n_total + col0) * R, u_bytes);
      const int kk = f0 + ahead_s * KS + 8 * tl.q;
      const uint32_t off = kk < R ? (uint32_t)tl.l * row_bytes + (uint32_t)kk * 2 : 0x80000000u;
#pragma unroll
      for (int c = 0; c < CB; ++c)
        u[c] = __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(ru, off + c * ROWS * row_bytes, 0, 0));
      advance(ahead, ahead_s);
      read_ahead();
    };
#pragma unroll
    for (int u = 0; u < kAdapterDepth; ++u) load_u(b[u]);
    while (at < count) {
#pragma unroll
      for (int u = 0; u < kAdapterDepth; ++u) {
        if (at >= count) break;
        uint32_t bits[RB];
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
          const uint32_t w = (uint32_t)__builtin_amdgcn_readfirstlane((int)words[rb * ROWS / 32]);
          bits[rb] = ROWS == 32 ? w : (w >> (rb * ROWS % 32)) & 0xFFFFu;
        }
#pragma unroll
        for (int c = 0; c < CB; ++c) {
          const bool bad = nonfinite(b[u][c]);
          const uint64_t broken = __ballot(bad);
          if (broken != 0) {
            b[u][c] = keep_or_zero(b[u][c], !bad);
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) acc[rb][c] = adapter_blow<ROWS>(broken, tl.mine(bits[rb]), acc[rb][c]);
          }
        }
        const uint8_t* t_at = lds + s * ad.parts * 256 * PIECES * 16;
        advance(at, s);
        read_words();
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
          if (bits[rb] == 0) continue;
          for (int p = 0; p < ad.parts; ++p) {
            const bf16x8 t =
                *reinterpret_cast<const bf16x8*>(t_at + ((p * 256 + rb * ROWS + tl.l) * PIECES + tl.q) * 16);
            const bf16x8 a = keep_or_zero(t, tl.mine(bits[rb]));
#pragma unroll
            for (int c = 0; c < CB; ++c) acc[rb][c] = adapter_mfma(a, b[u][c], acc[rb][c]);
          }
        }
        load_u(b[u]);
      }
    }
    __syncthreads();                                           // T's LDS is free
  }
}

// ---------------------------------------------------------------------------
// At most 64 rows.  The workgroup adds T's chunks up into LDS once
// (AdapterStage) as bf16 parts; its K-split waves share out the distinct
// adapters, and the first two adapters' U of each wave are loaded before the
// K loop (adapter_first) and used behind it.  Bound by latencies: 16 x 15360 x
// 5120 with 16 adapters of rank 16 takes 25.5 us where the product alone takes
// 18.8, 37 x 5120 x 13824 at rank 64 60 us and 50.
// ---------------------------------------------------------------------------
constexpr size_t adapter_stage_bytes(int rows) { return (size_t)kAdapterMaxParts * rows * 128 * 2; }

// Loads complete in the order they are issued, so what a wave needs first it
// has to load first: the row ids and the first T values (begin) go out ahead
// of the kernel's own loads, and U, which is needed last, behind them.
struct AdapterStage {
  int id;                                                     // of row `lane`
  f32x4 lo[kAdapterMaxChunks], hi[kAdapterMaxChunks];

  __device__ __forceinline__ void load(const AdapterArgs& ad, int m, int R, int i) {
    const float* p = ad.t + (int64_t)i * 8;                   // T is dense: row i / (R / 8), column 8 (i % (R / 8))
#pragma unroll
    for (int c = 0; c < kAdapterMaxChunks; ++c) {
      if (c >= ad.chunks) break;
      const float* pc = p + (int64_t)c * m * R;
      lo[c] = *reinterpret_cast<const f32x4*>(pc);
      hi[c] = *reinterpret_cast<const f32x4*>(pc + 4);
    }
  }
  __device__ __forceinline__ void write(const AdapterArgs& ad, int m, int R, int i, __bf16* lds) {
    float t[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      t[e] = lo[0][e];
      t[4 + e] = hi[0][e];
    }
#pragma unroll
    for (int c = 1; c < kAdapterMaxChunks; ++c) {
      if (c >= ad.chunks) break;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        t[e] += lo[c][e];
        t[4 + e] += hi[c][e];
      }
    }
    for (int part = 0; part < ad.parts; ++part)
      *reinterpret_cast<u32x4*>(lds + ((int64_t)part * m * R + i * 8)) = take_part(t);
  }
  __device__ __forceinline__ void begin(const AdapterArgs& ad, int m, int R, bool early, int tid) {
    id = adapter_of(ad.rows, ad.count, threadIdx.x & 63, m);
    if (early) load(ad, m, R, min(tid, m * (R / 8) - 1));
  }
  // T's parts to lds; started: begin loaded the thread's first values
  __device__ __forceinline__ void finish(const AdapterArgs& ad, int m, int R, bool started, __bf16* lds, int tid,
                                         int n) {
    for (int i = tid; i < m * (R / 8); i += n) {
      if (!started || i != tid) load(ad, m, R, i);
      write(ad, m, R, i, lds);
    }
  }
};

// The first adapters whose U a wave loads ahead, and how many 32-wide steps of
// their rank: one column block leaves registers for four adapters of rank 64,
// four blocks for two of rank 32.
template <int CB>
struct AdapterFirst {
  static constexpr int kAhead = CB == 1 ? 4 : 2, kSteps = CB <= 2 ? 2 : 1;
  int adapter[kAhead];                     // -1: none
  uint64_t match[kAhead];
  bf16x8 b[kAhead][kSteps][CB];            // U of columns n[c]
};

template <int CB>
__device__ __forceinline__ void adapter_u(const AdapterArgs& ad, int adapter, int n_total, int R, const int (&n)[CB],
                                          int j0, bf16x8 (&b)[CB]) {
  const int kk = j0 + 8 * (int)((threadIdx.x & 63) >> 4);
#pragma unroll
  for (int c = 0; c < CB; ++c) {
    const __bf16* up = ad.up + ((int64_t)adapter * n_total + n[c]) * R;
    b[c] = keep_or_zero(*reinterpret_cast<const bf16x8*>(up + min(kk, R - 8)), kk < R);
  }
}

// Wave `share` of `shares` takes the distinct adapters share, share + shares, ...
template <int CB>
__device__ __forceinline__ void adapter_first(const AdapterArgs& ad, int row_id, int n_total, int R,
                                              const int (&n)[CB], int share, int shares, AdapterFirst<CB>& first) {
  using F = AdapterFirst<CB>;
  const int id[1] = {row_id};
  AdapterWalk<1> walk(id);
  int d = -1;
#pragma unroll
  for (int i = 0; i < F::kAhead; ++i) {
    first.adapter[i] = -1;
    first.match[i] = 0;
    while (walk.next(id)) {
      if (++d % shares != share) continue;
      first.adapter[i] = walk.adapter;
      first.match[i] = walk.match[0];
      break;
    }
    if (first.adapter[i] < 0) continue;
#pragma unroll
    for (int s = 0; s < F::kSteps; ++s)
      if (s == 0 || 32 * s < R) adapter_u<CB>(ad, first.adapter[i], n_total, R, n, 32 * s, first.b[i][s]);
  }
}

// acc += one adapter's step from j0 on for the rows `match`, T's parts in LDS.
template <int RB, int CB>
__device__ __forceinline__ void adapter_step(const AdapterArgs& ad, int m, int R, uint64_t match, int j0,
                                             const bf16x8 (&b)[CB], const __bf16* lds, f32x4 (&acc)[RB][CB]) {
  const int lane = threadIdx.x & 63, lr = lane & 15, lq = lane >> 4;
  const int kk = j0 + 8 * lq, kc = min(kk, R - 8);
#pragma unroll
  for (int rb = 0; rb < RB; ++rb) {
    const uint32_t mask = (uint32_t)(match >> (16 * rb)) & 0xFFFFu;
    if (mask == 0) continue;
    f32x4 sum[CB];
#pragma unroll
    for (int c = 0; c < CB; ++c) sum[c] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int p = 0; p < ad.parts; ++p) {
      const bf16x8 a = keep_or_zero(
          *reinterpret_cast<const bf16x8*>(lds + ((int64_t)p * m + min(rb * 16 + lr, m - 1)) * R + kc),
          kk < R && ((mask >> lr) & 1));
#pragma unroll
      for (int c = 0; c < CB; ++c) sum[c] = adapter_mfma(a, b[c], sum[c]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool mine = (mask >> (4 * lq + i)) & 1;
#pragma unroll
      for (int c = 0; c < CB; ++c) acc[rb][c][i] += mine ? sum[c][i] : 0.0f;
    }
  }
}

template <int RB, int CB>
__device__ __forceinline__ void adapter_rows16(const AdapterArgs& ad, int m, int n_total, int R, const int (&n)[CB],
                                               int share, int shares, const AdapterFirst<CB>& first,
                                               const __bf16* lds, f32x4 (&acc)[RB][CB]) {
  using F = AdapterFirst<CB>;
#pragma unroll
  for (int i = 0; i < F::kAhead; ++i) {
    if (first.adapter[i] < 0) return;
#pragma unroll
    for (int s = 0; s < F::kSteps; ++s)
      if (s == 0 || 32 * s < R) adapter_step<RB, CB>(ad, m, R, first.match[i], 32 * s, first.b[i][s], lds, acc);
    for (int j0 = 32 * F::kSteps; j0 < R; j0 += 32) {
      bf16x8 b[CB];
      adapter_u<CB>(ad, first.adapter[i], n_total, R, n, j0, b);
      adapter_step<RB, CB>(ad, m, R, first.match[i], j0, b, lds, acc);
    }
  }
  const int id[1] = {adapter_of(ad.rows, ad.count, threadIdx.x & 63, m)};
  AdapterWalk<1> walk(id);
  for (int d = 0; walk.next(id); ++d) {
    if (d % shares != share || d < shares * F::kAhead) continue;
    for (int j0 = 0; j0 < R; j0 += 32) {
      bf16x8 b[CB];
      adapter_u<CB>(ad, walk.adapter, n_total, R, n, j0, b);
      adapter_step<RB, CB>(ad, m, R, walk.match[0], j0, b, lds, acc);
    }
  }
}

// ---------------------------------------------------------------------------
// T = s_a X D_a^T, as T^T = D_a X^T.  Workgroup (b, z, c, p): 16 RR rows, the
// row block's distinct adapters z, z + Z, ..., K chunk c (gpc groups of 128),
// rank blocks of 16 from p RBLK on.  Its NW waves take runs of the chunk in
// steps of 64 inputs and are summed through LDS in wave order.
// A step's rows (X's and D's, 128 bytes each) go HBM -> LDS with buffer_load
// ... lds, eight whole lines per instruction, into the wave's own two stages;
// the operands are read back from there.  (Loaded straight into the operand
// layout, neighbouring lanes read different rows, 16 bytes of a line each, and
// the line accesses bound the kernel: 32760 x 5120 at rank 32 took 128 us, with
// the rows read once more 222.)  Row r's 16-byte piece c sits in slot
// c ^ (r & 7), so that the operand reads spread over the banks.
// Rows without an adapter are not written (no product reads them).  32760 x
// 5120 at rank 32: 92 to 97 us (335 MB, 3.5 TB/s); 4096 rows at rank 16: 11.4.
//   PARTS: one chunk; T's bf16 parts to t16 (parts x m x r)
//   else:  the chunk's float32 sums to part (chunks x m x r)
// ---------------------------------------------------------------------------
struct AdapterDown {
  const __bf16* x;          // m x k
  const __bf16* down;       // count x r x k
  const float* scales;      // count
  const int* rows;          // m
  float* part;
  __bf16* t16;
  int m, k, r, count, chunks, gpc, parts;
  int z;                    // workgroups per row block
  int rank_parts;           // workgroups along the rank
  int run;                  // row blocks in a row before the next z; 0: all (z in blockIdx.z)
};

// Waves per workgroup: at most 8, and no more than leave room for a second
// workgroup on the compute unit (two stages of 2 KB per row block and wave;
// 16 waves with one row block each took 13.4 us where 8 take 11.2).
constexpr int adapter_down_waves(int rr, int rblk) { return 20 / (rr + rblk) < 8 ? 20 / (rr + rblk) : 8; }

template <int RBLK, int RR, bool PARTS>
__global__ __launch_bounds__(64 * adapter_down_waves(RR, RBLK)) void adapter_down_kernel(AdapterDown a) {
  constexpr int NW = adapter_down_waves(RR, RBLK);
  constexpr int ROWS = 16 * (RR + RBLK), STAGE = ROWS * 128;           // bytes of a step
  static_assert(RR <= 4 && RBLK <= 4, "one row id per lane; stages and partial tiles in LDS");
  static_assert(RR * RBLK * 1024 <= STAGE, "the partial tiles fit the first stages");
  __shared__ __attribute__((aligned(1024))) uint8_t st0[NW][STAGE];
  __shared__ __attribute__((aligned(1024))) uint8_t st1[NW][STAGE];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  const int lr = lane & 15, lq = lane >> 4;
  const int m = a.m, k = a.k, r = a.r;
  int block = blockIdx.x, z = blockIdx.z / a.rank_parts;
  if (a.run > 0) {
    const int runs = blockIdx.x / a.run;
    z = runs % a.z;
    block = runs / a.z * a.run + (blockIdx.x - runs * a.run);
  }
  const int m0 = block * 16 * RR;
  if (m0 >= m) return;
  const int r0 = blockIdx.z % a.rank_parts * 16 * RBLK;
  const int kb = blockIdx.y * a.gpc * kGroup;               // chunk start (< k)
  const int kl = min(a.gpc * kGroup, k - kb);
  const int id[1] = {lane < 16 * RR ? adapter_of(a.rows, a.count, m0 + lane, m) : -1};
  // this wave's steps of the chunk: a run of its own
  const int s0 = wave * (kl / 64) / NW, s1 = (wave + 1) * (kl / 64) / NW;
  const uint32_t row_bytes = (uint32_t)k * 2;
  // rows past M and ranks past r lie past their resource: zeros
  const rsrc_t rx = make_rsrc(a.x + (int64_t)m0 * k, (uint32_t)min(16 * RR, m - m0) * row_bytes);
  const uint32_t piece = (uint32_t)((lane & 7) ^ (lane >> 3)) * 16;    // of row lane / 8 (rows 8 i + lane / 8)
  const uint32_t lane_off = (uint32_t)(lane >> 3) * row_bytes + piece;
  uint32_t at[2];                                           // this lane's operand halves within a row block
#pragma unroll
  for (int h = 0; h < 2; ++h) at[h] = (uint32_t)(lr * 128 + (((2 * lq + h) ^ (lr & 7)) * 16));

  AdapterWalk<1> walk(id);
  for (int d = 0; walk.next(id); d = d + 1 == a.z ? 0 : d + 1) {
    if (d != z) continue;
    const rsrc_t rd = make_rsrc(a.down + ((int64_t)walk.adapter * r + r0) * k, (uint32_t)min(16 * RBLK, r - r0) * row_bytes);
    f32x4 acc[RR][RBLK];
#pragma unroll
    for (int i = 0; i < RR; ++i)
#pragma unroll
      for (int j = 0; j < RBLK; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    // step st into a stage; past the run, its first step again (not used)
    auto issue = [&](uint8_t* stage, int st) __attribute__((always_inline)) {
      const uint32_t soff = (uint32_t)(kb + 64 * (st < s1 ? st : s0)) * 2;
#pragma unroll
      for (int i = 0; i < 2 * RR; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_ptr_t)(stage + i * 1024), 16,
                                                 lane_off + (uint32_t)(8 * i) * row_bytes, soff, 0, 0);
#pragma unroll
      for (int i = 0; i < 2 * RBLK; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rd, (lds_ptr_t)(stage + (2 * RR + i) * 1024), 16,
                                                 lane_off + (uint32_t)(8 * i) * row_bytes, soff, 0, 0);
    };
    auto compute = [&](const uint8_t* stage) __attribute__((always_inline)) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        bf16x8 bv[RR], av[RBLK];
#pragma unroll
        for (int i = 0; i < RR; ++i) bv[i] = *reinterpret_cast<const bf16x8*>(stage + i * 2048 + at[h]);
#pragma unroll
        for (int j = 0; j < RBLK; ++j) av[j] = *reinterpret_cast<const bf16x8*>(stage + (RR + j) * 2048 + at[h]);
#pragma unroll
        for (int i = 0; i < RR; ++i)
#pragma unroll
          for (int j = 0; j < RBLK; ++j) acc[i][j] = mfma16x16x32(av[j], bv[i], acc[i][j]);
      }
    };
    constexpr int NI = 2 * (RR + RBLK);                     // loads of a step
    // all but the last step's loads have landed (the fence keeps the reads below)
    auto landed = [&] {
      __builtin_amdgcn_s_waitcnt(0x0F70 | (NI & 15) | ((NI >> 4) << 14));
      asm volatile("" ::: "memory");
    };
    // this wave's reads of a stage are done before loads overwrite it
    auto read = [&] {
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(0xC07F);
    };
    if (s0 < s1) {
      issue(&st0[wave][0], s0);
      for (int st = s0; st < s1; st += 2) {
        read();
        issue(&st1[wave][0], st + 1);
        landed();
        compute(&st0[wave][0]);
        if (st + 1 >= s1) break;
        read();
        issue(&st0[wave][0], st + 2);
        landed();
        compute(&st1[wave][0]);
      }
    }
    // the partial tiles go where the first stages were
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    f32x4* red = reinterpret_cast<f32x4*>(&st0[0][0]);      // [wave][row block][rank block][lane]
#pragma unroll
    for (int i = 0; i < RR; ++i)
#pragma unroll
      for (int j = 0; j < RBLK; ++j) red[((wave * RR + i) * RBLK + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    const float s = a.scales[walk.adapter];
    // the tiles (row block i, rank block j) go round the waves; partial sums in wave order
    for (int tile = wave; tile < RR * RBLK; tile += NW) {
      const int i = tile / RBLK, j = tile - i * RBLK;
      f32x4 v = red[tile * 64 + lane];
#pragma unroll
      for (int w = 1; w < NW; ++w) {
        const f32x4 o = red[(w * RR * RBLK + tile) * 64 + lane];
        v[0] += o[0]; v[1] += o[1]; v[2] += o[2]; v[3] += o[3];
      }
      v[0] *= s; v[1] *= s; v[2] *= s; v[3] *= s;
      const int mm = m0 + 16 * i + lr;
      const int rr = r0 + j * 16 + 4 * lq;   // rows rr .. rr+3 of T^T; r % 8 == 0, so rr < r implies rr + 3 < r
      if (!((walk.match[0] >> (16 * i + lr)) & 1) || rr >= r) continue;
      if constexpr (PARTS) {
        for (int p = 0; p < a.parts; ++p) {
          const u32x2 w = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
          *reinterpret_cast<u32x2*>(a.t16 + ((int64_t)p * m + mm) * r + rr) = w;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            v[2 * e] -= bf16_bits_to_f32(w[e] & 0xFFFFu);
            v[2 * e + 1] -= __builtin_bit_cast(float, w[e] & 0xFFFF0000u);
          }
        }
      } else {
        *reinterpret_cast<f32x4*>(a.part + ((int64_t)blockIdx.y * m + mm) * r + rr) = v;
      }
    }
    __syncthreads();                         // the stages are free for the next adapter
  }
}

}  // namespace ddg
