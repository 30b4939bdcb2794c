// Low-rank adapters of many requests beside one shared product: row i of Y
// also gets s_a T_i U_a^T with a = rows[i] and T_i = X_i D_a^T.
//
//   adapter_down_kernel  T (times s_a) in float32, K in `chunks` parts whose
//                        sums the product adds up, in order;
//   adapter_tile32 / adapter_tile16 / adapter_rows16
//                        the branch inside the product kernels: the first
//                        terms of their accumulators.
//
// A block of rows may mix adapters.  Every wave walks the distinct adapters of
// its rows (ballots over the ids held one row per lane, so the walk is uniform
// over the wave) and runs the matrix instructions of one adapter for the row
// blocks that hold it, with the other rows' T as zeros.  Requests are runs of
// rows, so most blocks hold one adapter and cost what one shared adapter does.
// A block that mixes adapters adds each adapter's sums to that adapter's rows
// only: an infinity or NaN among its weights reaches no other request.
//
// T is float32 and enters the bf16 matrix instructions as a sum of bf16
// parts: two (to 2^-16 of T) for a bf16 Y, whose own
// rounding is 2^-8, and three (to 2^-24) for a float32 Y.  The products of
// bf16 parts are exact in the float32 accumulator, so Y is rounded once.
#pragma once

#include "ddg_device.hpp"

namespace ddg {

struct AdapterArgs {
  const int* rows;          // M adapter numbers; outside [0, count): no adapter
  const float* t;           // chunks x M x R
  const __bf16* up;         // count x N x R
  int count;
  int chunks;
};
struct NoAdapters {};       // a product without them

constexpr int kAdapterMaxChunks = 8;

// Row r's adapter, -1 for none and for rows past m.
__device__ __forceinline__ int adapter_of(const int* rows, int count, int r, int m) {
  const int id = r < m ? rows[r] : -1;
  return (unsigned)id < (unsigned)count ? id : -1;
}

// Eight values of T_row from column kc on, its chunks added in order.
__device__ __forceinline__ void adapter_t8(const AdapterArgs& ad, int row, int m, int R, int kc, float (&t)[8]) {
  const float* p = ad.t + (int64_t)row * R + kc;
  const int64_t chunk = (int64_t)m * R;
  const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    t[i] = a[i];
    t[4 + i] = b[i];
  }
  for (int c = 1; c < ad.chunks; ++c) {
    const f32x4 u = *reinterpret_cast<const f32x4*>(p + c * chunk);
    const f32x4 v = *reinterpret_cast<const f32x4*>(p + c * chunk + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      t[i] += u[i];
      t[4 + i] += v[i];
    }
  }
}

// The next bf16 part of t (nearest), which is taken off t.
__device__ __forceinline__ bf16x8 take_part(float (&t)[8]) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = pack_bf16x2(t[2 * i], t[2 * i + 1]);
    t[2 * i] -= bf16_bits_to_f32(w[i] & 0xFFFFu);
    t[2 * i + 1] -= __builtin_bit_cast(float, w[i] & 0xFFFF0000u);
  }
  return __builtin_bit_cast(bf16x8, w);
}

__device__ __forceinline__ f32x16 adapter_mfma(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 adapter_mfma(bf16x8 a, bf16x8 b, f32x4 c) { return mfma16x16x32(a, b, c); }

// Distinct adapters of up to 64 W rows (id[j]: row 64 j + lane), one at a time.
template <int W>
struct AdapterWalk {
  uint64_t pending[W], match[W];
  int adapter;
  __device__ __forceinline__ explicit AdapterWalk(const int (&id)[W]) {
#pragma unroll
    for (int j = 0; j < W; ++j) pending[j] = __ballot(id[j] >= 0);
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

// One k-step of one adapter for a row block whose matching rows are `mask`:
// lane (row lr, k part q) holds t of its row; b[c] the adapter's columns.
template <int CB, typename Acc, typename RowOf>
__device__ __forceinline__ void adapter_block(float (&t)[8], const bf16x8 (&b)[CB], int parts, uint32_t mask,
                                              uint32_t full, Acc (&acc)[CB], RowOf row_of) {
  if (mask == full) {
    for (int p = 0; p < parts; ++p) {
      const bf16x8 a = take_part(t);
#pragma unroll
      for (int c = 0; c < CB; ++c) acc[c] = adapter_mfma(a, b[c], acc[c]);
    }
    return;
  }
  constexpr int N = sizeof(Acc) / 4;
  Acc sum[CB];
#pragma unroll
  for (int c = 0; c < CB; ++c)
#pragma unroll
    for (int i = 0; i < N; ++i) sum[c][i] = 0.0f;
  for (int p = 0; p < parts; ++p) {
    const bf16x8 a = take_part(t);
#pragma unroll
    for (int c = 0; c < CB; ++c) sum[c] = adapter_mfma(a, b[c], sum[c]);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const bool mine = (mask >> row_of(i)) & 1;
#pragma unroll
    for (int c = 0; c < CB; ++c) acc[c][i] += mine ? sum[c][i] : 0.0f;
  }
}

// The branch of a 256-row tile from row m0 for 32 columns (lane column n,
// clamped to the last), in the 32x32 accumulator layout.
__device__ __forceinline__ void adapter_tile32(const AdapterArgs& ad, int m, int n_total, int R, int parts, int m0,
                                               int n, f32x16 (&acc)[8]) {
  const int lane = threadIdx.x & 63, lr = lane & 31, lh = lane >> 5;
  const bf16x8 zero = __builtin_bit_cast(bf16x8, u32x4{0u, 0u, 0u, 0u});
  int id[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) id[j] = adapter_of(ad.rows, ad.count, m0 + 64 * j + lane, m);
  AdapterWalk<4> walk(id);
  while (walk.next(id)) {
    const __bf16* up = ad.up + ((int64_t)walk.adapter * n_total + n) * R;
    uint32_t mask[8];
#pragma unroll
    for (int rb = 0; rb < 8; ++rb) mask[rb] = (uint32_t)(walk.match[rb >> 1] >> (32 * (rb & 1)));
    for (int j0 = 0; j0 < R; j0 += 16) {
      const int kk = j0 + 8 * lh;
      const bool kok = kk < R;
      const int kc = min(kk, R - 8);
      const bf16x8 v = *reinterpret_cast<const bf16x8*>(up + kc);
      const bf16x8 b[1] = {kok ? v : zero};
      // four row blocks' loads in flight at a time (eight spill registers)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float t[4][8];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (mask[4 * half + i]) adapter_t8(ad, min(m0 + (4 * half + i) * 32 + lr, m - 1), m, R, kc, t[i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int rb = 4 * half + i;
          if (!mask[rb]) continue;
          const bool mine = kok && ((mask[rb] >> lr) & 1);
#pragma unroll
          for (int e = 0; e < 8; ++e) t[i][e] = mine ? t[i][e] : 0.0f;
          f32x16 a1[1] = {acc[rb]};
          adapter_block<1>(t[i], b, parts, mask[rb], 0xFFFFFFFFu, a1,
                           [&](int e) { return 8 * (e >> 2) + 4 * lh + (e & 3); });
          acc[rb] = a1[0];
        }
      }
    }
  }
}

// The branch of a 256-row tile from row m0 for three blocks of 16 columns
// (lane columns n[c], clamped to the last), in the 16x16 accumulator layout.
__device__ __forceinline__ void adapter_tile16(const AdapterArgs& ad, int m, int n_total, int R, int parts, int m0,
                                               const int (&n)[3], f32x4 (&acc)[16][3]) {
  const int lane = threadIdx.x & 63, lr = lane & 15, lq = lane >> 4;
  const bf16x8 zero = __builtin_bit_cast(bf16x8, u32x4{0u, 0u, 0u, 0u});
  int id[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) id[j] = adapter_of(ad.rows, ad.count, m0 + 64 * j + lane, m);
  AdapterWalk<4> walk(id);
  while (walk.next(id)) {
    const __bf16* up = ad.up + (int64_t)walk.adapter * n_total * R;
    for (int j0 = 0; j0 < R; j0 += 32) {
      const int kk = j0 + 8 * lq;
      const bool kok = kk < R;
      const int kc = min(kk, R - 8);
      bf16x8 b[3];
#pragma unroll
      for (int c = 0; c < 3; ++c) {
        const bf16x8 v = *reinterpret_cast<const bf16x8*>(up + (int64_t)n[c] * R + kc);
        b[c] = kok ? v : zero;
      }
#pragma unroll
      for (int part = 0; part < 4; ++part) {
        float t[4][8];
        uint32_t mask[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int rb = 4 * part + i;
          mask[i] = (uint32_t)(walk.match[rb >> 2] >> (16 * (rb & 3))) & 0xFFFFu;
          if (mask[i]) adapter_t8(ad, min(m0 + rb * 16 + lr, m - 1), m, R, kc, t[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (!mask[i]) continue;
          const bool mine = kok && ((mask[i] >> lr) & 1);
#pragma unroll
          for (int e = 0; e < 8; ++e) t[i][e] = mine ? t[i][e] : 0.0f;
          adapter_block<3>(t[i], b, parts, mask[i], 0xFFFFu, acc[4 * part + i], [&](int e) { return 4 * lq + e; });
        }
      }
    }
  }
}

// The branch of at most 64 rows for CB blocks of 16 columns (lane columns
// n[c]); of the distinct adapters, those numbered share, share + shares, ...
// (the caller's waves split them and add their accumulators up afterwards).
template <int RB, int CB>
__device__ __forceinline__ void adapter_rows16(const AdapterArgs& ad, int m, int n_total, int R, int parts,
                                               const int (&n)[CB], int share, int shares, f32x4 (&acc)[RB][CB]) {
  const int lane = threadIdx.x & 63, lr = lane & 15, lq = lane >> 4;
  const bf16x8 zero = __builtin_bit_cast(bf16x8, u32x4{0u, 0u, 0u, 0u});
  const int id[1] = {adapter_of(ad.rows, ad.count, lane, m)};
  AdapterWalk<1> walk(id);
  for (int d = 0; walk.next(id); d = d + 1 == shares ? 0 : d + 1) {
    if (d != share) continue;
    const __bf16* up = ad.up + (int64_t)walk.adapter * n_total * R;
    for (int j0 = 0; j0 < R; j0 += 32) {
      const int kk = j0 + 8 * lq;
      const bool kok = kk < R;
      const int kc = min(kk, R - 8);
      bf16x8 b[CB];
#pragma unroll
      for (int c = 0; c < CB; ++c) {
        const bf16x8 v = *reinterpret_cast<const bf16x8*>(up + (int64_t)n[c] * R + kc);
        b[c] = kok ? v : zero;
      }
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) {
        const uint32_t mask = (uint32_t)(walk.match[0] >> (16 * rb)) & 0xFFFFu;
        if (!mask) continue;
        float t[8];
        adapter_t8(ad, min(rb * 16 + lr, m - 1), m, R, kc, t);
        const bool mine = kok && ((mask >> lr) & 1);
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = mine ? t[e] : 0.0f;
        adapter_block<CB>(t, b, parts, mask, 0xFFFFu, acc[rb], [&](int e) { return 4 * lq + e; });
      }
    }
  }
}

// part[c][i][j] = s_a sum over chunk c's inputs of X[i][k] D_a[j][k], a the
// adapter of row i, as T^T = D_a X^T (both matrix operands then read 16
// consecutive bytes).  Workgroup (b, c, z): 16 RR rows, K chunk c (gpc groups
// of 128), the row block's distinct adapters z, z + gridDim.z, ...  Its waves
// split the chunk in steps of 32 and are summed through LDS in wave order.
// Rows without an adapter are not written (no product reads them).
constexpr int kAdapterWaves = 4;

template <int RBLK, int RR>
__global__ __launch_bounds__(64 * kAdapterWaves) void adapter_down_kernel(const __bf16* __restrict__ x,
                                                                          const __bf16* __restrict__ down,
                                                                          const float* __restrict__ scales,
                                                                          const int* __restrict__ rows, int count,
                                                                          float* __restrict__ part, int m, int k,
                                                                          int r, int gpc) {
  static_assert(RR * RBLK <= 8 && RR <= 4, "partial tiles in LDS: at most 32 KB; one row id per lane");
  constexpr int NW = kAdapterWaves;
  __shared__ f32x4 red[NW][RR][RBLK][64];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  const int lr = lane & 15, lq = lane >> 4;
  const int m0 = blockIdx.x * 16 * RR;
  const int kb = blockIdx.y * gpc * kGroup;                 // chunk start (< k)
  const int kl = min(gpc * kGroup, k - kb);
  const int id[1] = {lane < 16 * RR ? adapter_of(rows, count, m0 + lane, m) : -1};
  const __bf16* xrow[RR];
#pragma unroll
  for (int i = 0; i < RR; ++i) xrow[i] = x + (int64_t)min(m0 + 16 * i + lr, m - 1) * k + kb + 8 * lq;
  constexpr int LPS = RR + RBLK;                            // loads of one step
  constexpr int U = LPS <= 3 ? 8 : (LPS <= 5 ? 4 : 2);
  const int steps = (kl - wave * 32 + 32 * NW - 1) / (32 * NW);
  AdapterWalk<1> walk(id);
  for (int d = 0; walk.next(id); d = d + 1 == (int)gridDim.z ? 0 : d + 1) {
    if (d != (int)blockIdx.z) continue;
    const __bf16* da = down + (int64_t)walk.adapter * r * k + kb + 8 * lq;
    const __bf16* drow[RBLK];
#pragma unroll
    for (int j = 0; j < RBLK; ++j) drow[j] = da + (int64_t)min(j * 16 + lr, r - 1) * k;
    f32x4 acc[RR][RBLK];
#pragma unroll
    for (int i = 0; i < RR; ++i)
#pragma unroll
      for (int j = 0; j < RBLK; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    int st = 0;
    for (; st + U <= steps; st += U) {
      bf16x8 bv[U][RR], av[U][RBLK];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k0 = wave * 32 + 32 * NW * (st + u);
#pragma unroll
        for (int i = 0; i < RR; ++i) bv[u][i] = *reinterpret_cast<const bf16x8*>(xrow[i] + k0);
#pragma unroll
        for (int j = 0; j < RBLK; ++j) av[u][j] = *reinterpret_cast<const bf16x8*>(drow[j] + k0);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < RR; ++i)
#pragma unroll
          for (int j = 0; j < RBLK; ++j) acc[i][j] = mfma16x16x32(av[u][j], bv[u][i], acc[i][j]);
    }
    for (; st < steps; ++st) {
      const int k0 = wave * 32 + 32 * NW * st;
      bf16x8 b[RR];
#pragma unroll
      for (int i = 0; i < RR; ++i) b[i] = *reinterpret_cast<const bf16x8*>(xrow[i] + k0);
#pragma unroll
      for (int j = 0; j < RBLK; ++j) {
        const bf16x8 a = *reinterpret_cast<const bf16x8*>(drow[j] + k0);
#pragma unroll
        for (int i = 0; i < RR; ++i) acc[i][j] = mfma16x16x32(a, b[i], acc[i][j]);
      }
    }
#pragma unroll
    for (int i = 0; i < RR; ++i)
#pragma unroll
      for (int j = 0; j < RBLK; ++j) red[wave][i][j][lane] = acc[i][j];
    __syncthreads();
    const float s = scales[walk.adapter];
    // wave i (< RR) sums and stores row block i, the partials in wave order
#pragma unroll
    for (int i = 0; i < RR; ++i) {
      if (i != wave || !((walk.match[0] >> (16 * i + lr)) & 1)) continue;
      const int mm = m0 + 16 * i + lr;
#pragma unroll
      for (int j = 0; j < RBLK; ++j) {
        f32x4 v = red[0][i][j][lane];
#pragma unroll
        for (int w = 1; w < NW; ++w) {
          const f32x4 o = red[w][i][j][lane];
          v[0] += o[0]; v[1] += o[1]; v[2] += o[2]; v[3] += o[3];
        }
        const int rr = j * 16 + 4 * lq;      // rows rr .. rr+3 of T^T; r % 8 == 0, so rr < r implies rr + 3 < r
        if (rr < r) {
          v[0] *= s; v[1] *= s; v[2] *= s; v[3] *= s;
          *reinterpret_cast<f32x4*>(part + ((int64_t)blockIdx.y * m + mm) * r + rr) = v;
        }
      }
    }
    __syncthreads();                         // red is free for the next adapter
  }
}

}  // namespace ddg
