// Rotary positions, alone or behind the norms of queries and keys.
//
// A head is a row x of D values.  Its first 2P values are P pairs (u, v):
// (x[2p], x[2p+1]) in the interleaved layout, (x[p], x[P+p]) in the half
// layout.  Pair p turns by the angle theta = pos[axis(p)] * freq[p]:
//   (u, v) -> amplitude * (u cos theta - v sin theta, v cos theta + u sin theta),
// the inverse by -theta; values from 2P on pass through.  With a norm, x is
// first replaced by x * rsqrt(mean(x^2) + eps) * w, the mean over the head
// or over all heads of the token.  Everything between the load and the one
// rounding at the store is float32; the angle is float64 (a position of 10^6
// times a frequency near 1 leaves float32 no fraction of a turn to speak of).
//
// Bound by HBM: each value is read and written once (bf16: norm per head and
// rotation of 32760 tokens of 40 + 40 heads of 128 266 us, 5.0 TB/s; rotation
// alone of 32768 tokens of 24 heads 83 us, 4.8 TB/s; a large copy reaches 5.3
// to 5.6), with few tokens by the launch (one token 3.8 us).  The sines and cosines
// belong to a (token, pair) and not to a head, so a wave computes those of its
// lanes' pairs once per token and keeps them in registers over the heads; no
// table is read.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "ddg.h"
#include "ddg_launch.hpp"

namespace ddg {

namespace {

// cos and sin of 2 pi t: whole turns drop out in float64 and the rest is
// taken to the nearest quarter turn, so that the Taylor sums below run over
// at most pi/4 (their first dropped terms are 2e-9 of x for the sine and
// 1e-10 for the cosine, under half an ulp of float32).
__device__ __forceinline__ void cos_sin_turns(double t, float& c, float& s) {
  t -= __builtin_rint(t);
  const double q = __builtin_rint(4.0 * t);
  const float x = (float)(__builtin_fma(-0.25, q, t) * 6.283185307179586477);
  const float z = x * x;
  float ps = __builtin_fmaf(z, 1.0f / 362880.0f, -1.0f / 5040.0f);
  ps = __builtin_fmaf(z, ps, 1.0f / 120.0f);
  ps = __builtin_fmaf(z, ps, -1.0f / 6.0f);
  const float sx = __builtin_fmaf(x * z, ps, x);
  float pc = __builtin_fmaf(z, -1.0f / 3628800.0f, 1.0f / 40320.0f);
  pc = __builtin_fmaf(z, pc, -1.0f / 720.0f);
  pc = __builtin_fmaf(z, pc, 1.0f / 24.0f);
  pc = __builtin_fmaf(z, pc, -0.5f);
  const float cx = __builtin_fmaf(z, pc, 1.0f);
  const int n = (int)q;                              // -2 .. 2 quarter turns
  const float a = (n & 1) ? sx : cx, b = (n & 1) ? cx : sx;
  c = ((n + 1) & 2) ? -a : a;
  s = (n & 2) ? -b : b;
}

// Angle of pair p at the token whose positions start at pos, in turns.
__device__ __forceinline__ double pair_turns(const RopeArgs& a, const int32_t* pos, int p) {
  int axis = 0;
#pragma unroll
  for (int i = 0; i < kRopeMaxAxes - 1; ++i) axis += p >= a.ends[i] ? 1 : 0;
  return (double)pos[axis] * (a.freqs[p] * 0.15915494309189533577);
}

// V consecutive values of a row as loaded (the address is a multiple of their
// bytes), and their conversion.
template <typename T, int V>
struct Chunk {
  static constexpr int W = sizeof(T) * V / 4 > 0 ? (int)sizeof(T) * V / 4 : 1;     // dwords
  uint32_t w[W];
  __device__ __forceinline__ void load(const void* base, int64_t i) {
    const T* p = static_cast<const T*>(base) + i;
    if constexpr (sizeof(T) * V == 16) {
      const u32x4 t = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = t[j];
    } else if constexpr (sizeof(T) * V == 8) {
      const u32x2 t = *reinterpret_cast<const u32x2*>(p);
      w[0] = t[0];
      w[1] = t[1];
    } else if constexpr (sizeof(T) * V == 4) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
      w[0] = *reinterpret_cast<const uint16_t*>(p);
    }
  }
  // the words as they are: values() after it converts again, where the
  // compiler would keep the first conversion's twice as many registers
  __device__ __forceinline__ void keep() {
#pragma unroll
    for (int j = 0; j < W; ++j) asm("" : "+v"(w[j]));
  }
  __device__ __forceinline__ void values(float (&f)[V]) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int j = 0; j < V; ++j) f[j] = __builtin_bit_cast(float, w[j]);
    } else if constexpr (V == 1) {
      f[0] = bf16_bits_to_f32(w[0]);
    } else {
#pragma unroll
      for (int j = 0; j < V / 2; ++j) {
        f[2 * j] = bf16_bits_to_f32(w[j] & 0xFFFFu);
        f[2 * j + 1] = __builtin_bit_cast(float, w[j] & 0xFFFF0000u);
      }
    }
  }
};

template <typename T, int V>
__device__ __forceinline__ void store_vals(void* base, int64_t i, const float (&f)[V]) {
  T* p = static_cast<T*>(base) + i;
  if constexpr (sizeof(T) == 4 && V == 4) {
    *reinterpret_cast<f32x4*>(p) = f32x4{f[0], f[1], f[2], f[3]};
  } else if constexpr (sizeof(T) == 2 && V == 8) {
    *reinterpret_cast<u32x4*>(p) = u32x4{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                                         pack_bf16x2(f[6], f[7])};
  } else if constexpr (sizeof(T) == 2 && V == 4) {
    *reinterpret_cast<u32x2*>(p) = u32x2{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3])};
  } else if constexpr (sizeof(T) == 4 && V == 2) {
    *reinterpret_cast<f32x2*>(p) = f32x2{f[0], f[1]};
  } else if constexpr (sizeof(T) == 2 && V == 2) {
    *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(f[0], f[1]);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) p[j] = (T)f[j];
  }
}

// V norm weights from entry i on (1 without weights); vec: 16-byte aligned
// and i a multiple of V.
template <int V>
__device__ __forceinline__ void load_weight(const RopeTensor& x, bool w_f32, int64_t i, float (&f)[V]) {
  if (x.w == nullptr) {
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] = 1.0f;
  } else if (w_f32) {
    const float* p = static_cast<const float*>(x.w) + i;
    if (V >= 4 && x.w_vec) {
#pragma unroll
      for (int j = 0; j < V / 4; ++j) {
        const f32x4 t = *reinterpret_cast<const f32x4*>(p + 4 * j);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[4 * j + e] = t[e];
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) f[j] = p[j];
    }
  } else if (V >= 4 && x.w_vec) {
    Chunk<__bf16, V> t;
    t.load(x.w, i);
    t.values(f);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] = bf16_bits_to_f32(static_cast<const uint16_t*>(x.w)[i + j]);
  }
}

// A slot is two chunks of V values of a head: chunk a and chunk b.  Slots
// below P / V hold the rotated part: chunk a at V slot, chunk b P further on,
// so that in the half layout the pairs are (a[j], b[j]) and in the
// interleaved one lie inside the chunks (V = 1: the pair itself).  The other
// slots hold the rest of the head in the same way, its first half and its
// second.  P and D / 2 are multiples of V.
template <int V, bool HALF>
struct Slot {
  int ia, ib;
  bool turns;
  __device__ __forceinline__ Slot(const RopeArgs& a, int slot) {
    turns = slot * V < a.pairs;
    if (!turns) {
      ia = a.pairs + slot * V;
      ib = a.dim / 2 + slot * V;
    } else if (V == 1 && !HALF) {
      ia = 2 * slot;
      ib = ia + 1;
    } else {
      ia = slot * V;
      ib = a.pairs + ia;
    }
  }
  // the pair whose angle entry j of the slot's V angles is
  __device__ __forceinline__ int pair(int slot, int j) const {
    if (HALF || V == 1) return slot * V + j;
    return j < V / 2 ? ia / 2 + j : ib / 2 + j - V / 2;
  }
};

template <int V, bool HALF>
__device__ __forceinline__ void turn_slot(float (&fa)[V], float (&fb)[V], const float (&c)[V], const float (&s)[V]) {
  if constexpr (HALF || V == 1) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float u = fa[j], v = fb[j];
      fa[j] = __builtin_fmaf(u, c[j], -(v * s[j]));
      fb[j] = __builtin_fmaf(v, c[j], u * s[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < V / 2; ++j) {
      const float u = fa[2 * j], v = fa[2 * j + 1];
      fa[2 * j] = __builtin_fmaf(u, c[j], -(v * s[j]));
      fa[2 * j + 1] = __builtin_fmaf(v, c[j], u * s[j]);
      const float u2 = fb[2 * j], v2 = fb[2 * j + 1];
      const float c2 = c[V / 2 + j], s2 = s[V / 2 + j];
      fb[2 * j] = __builtin_fmaf(u2, c2, -(v2 * s2));
      fb[2 * j + 1] = __builtin_fmaf(v2, c2, u2 * s2);
    }
  }
}

template <int M>
__device__ __forceinline__ float add_dpp(float v) {
  return v + __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), M, 0xF, 0xF, true));
}

// Sum over each aligned run of 2^lg lanes, the same in all of them.  Once
// the lanes of a quad (a half row) agree, a mirror adds the other quad (half).
__device__ __forceinline__ float run_sum(float v, int lg) {
  if (lg > 0) v = add_dpp<0xB1>(v);       // lane ^ 1
  if (lg > 1) v = add_dpp<0x4E>(v);       // lane ^ 2
  if (lg > 2) v = add_dpp<0x141>(v);      // half-row mirror
  if (lg > 3) v = add_dpp<0x140>(v);      // row mirror
  if (lg > 4) v += __shfl_xor(v, 16);
  if (lg > 5) v += __shfl_xor(v, 32);
  return v;
}

// 1 / sqrt(v): the hardware's estimate (within an ulp) and one Newton step,
// the library's root where the step could leave the normal range.
__device__ __forceinline__ float rsqrt_of(float v) {
  if (!(v > 0x1p-100f && v < 0x1p100f)) return 1.0f / __builtin_sqrtf(v);
  const float y = __builtin_amdgcn_rsqf(v);
  const float h = __builtin_fmaf(-v * y, y, 1.0f);             // 1 - v y^2
  return __builtin_fmaf(0.5f * y, h, y);
}

constexpr int kRopeWaves = 4;

// A token's cosines and sines, one pair per lane (all of a wave's lanes at
// once would compute each pair once per head group, 8 times at 128 values per
// head), handed to the lanes that need them through the wave's own LDS.
struct WaveAngles {
  __attribute__((aligned(16))) float c[kRopeMaxHeadDim / 2], s[kRopeMaxHeadDim / 2];
  __device__ __forceinline__ void fill(const RopeArgs& a, const int32_t* pos, int lane, int at) {
    for (int p = lane; p < a.pairs; p += 64) {
      float cp, sp;
      cos_sin_turns(pair_turns(a, pos, p), cp, sp);
      c[at + p] = cp * a.amplitude;
      s[at + p] = sp * a.signed_amplitude;
    }
  }
  __device__ __forceinline__ void filled() const {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
  __device__ __forceinline__ void compute(const RopeArgs& a, const int32_t* pos, int lane) {
    fill(a, pos, lane, 0);
    filled();
  }
  // at: the token's first pair
  template <int V, bool HALF>
  __device__ __forceinline__ void take(const Slot<V, HALF>& k, int slot, float (&fc)[V], float (&fs)[V],
                                       int at = 0) const {
    // runs of R consecutive pairs, aligned to R
    constexpr int R = HALF || V == 1 ? (V < 4 ? V : 4) : V / 2;
    typedef float run __attribute__((ext_vector_type(R)));
#pragma unroll
    for (int j = 0; j < V; j += R) {
      const int p = at + k.pair(slot, j);
      const run rc = *reinterpret_cast<const run*>(c + p), rs = *reinterpret_cast<const run*>(s + p);
#pragma unroll
      for (int e = 0; e < R; ++e) {
        fc[j + e] = rc[e];
        fs[j + e] = rs[e];
      }
    }
  }
};

// No norm, or the norm over each head.  A wave takes one token (or, with
// splits > 1, one of `splits` shares of its heads): 2^lg lanes per head, one
// slot per lane, 64 >> lg heads at a time, query heads first.  V = 1 gives a
// head to the whole wave, up to NS slots per lane.  The next heads' values
// are loaded before the current ones are turned, the first ones before the
// angles are computed.  The norm weights go through LDS once per workgroup:
// loaded by every lane where it needs them, q's and k's were four latencies
// in a row.  Where q and k have few heads, PACK gives a wave's lanes to several
// tokens, as many as keep the heads' lanes busy and their angles in LDS: a
// vector instruction costs the same for 8 lanes as for 64, and with 1 + 1
// heads those outweigh the bytes (33610 tokens of 1 + 1 heads of 128: 41 us
// without, 20 with).
template <typename T, int V, bool HALF, bool NORM, bool PACK>
__global__ __launch_bounds__(64 * kRopeWaves) void rope_head_kernel(RopeArgs a) {
  constexpr int NS = V == 1 ? kRopeMaxHeadDim / 128 : 1;
  __shared__ WaveAngles ang[kRopeWaves];
  __shared__ __attribute__((aligned(16))) float weights[NORM ? 2 * kRopeMaxHeadDim : 1];     // q's, k's
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // PACK: hpw heads of each of 1 << lt tokens at a time
  const int lt = PACK ? a.lt : 0, hpw = 64 >> (a.lg + lt);
  const int sl = lane & ((1 << a.lg) - 1), hl = (lane >> a.lg) & (hpw - 1), tk = PACK ? lane / (hpw << a.lg) : 0;
  const int slots = a.dim / (2 * V);
  constexpr int WL = 2 * kRopeMaxHeadDim / (64 * kRopeWaves);                               // per lane
  float w_mine[WL];
  if constexpr (NORM) {
#pragma unroll
    for (int i = 0; i < WL; ++i) {
      const int at = threadIdx.x + i * 64 * kRopeWaves, e = min(at % kRopeMaxHeadDim, a.dim - 1);
      load_weight<1>(at < kRopeMaxHeadDim ? a.q : a.k, a.w_f32, e, reinterpret_cast<float(&)[1]>(w_mine[i]));
    }
  }
  bool weights_there = !NORM;
  const int gq = (a.q.heads + hpw - 1) / hpw, gk = (a.k.heads + hpw - 1) / hpw, groups = gq + gk;
  const int rows = a.batch * a.tokens;
  const int64_t total = PACK ? ((int64_t)rows + (1 << lt) - 1) >> lt : (int64_t)rows * a.splits;
  const float inv_dim = 1.0f / (float)a.dim;
  for (int64_t w0 = (int64_t)blockIdx.x * kRopeWaves; w0 < total; w0 += (int64_t)gridDim.x * kRopeWaves) {
    // past the last wave's work: its work again, not stored (every wave
    // reaches the barrier)
    bool live = w0 + wave < total;
    const int64_t w = live ? w0 + wave : total - 1;
    int row = (int)w, part = 0, g0 = 0, g1 = groups;
    if constexpr (PACK) {
      const int64_t mine = (w << lt) + tk;
      live = live && mine < rows;
      row = (int)min(mine, (int64_t)rows - 1);
    } else if (a.splits > 1) {                         // total < 2^31
      row = (int)w / a.splits;
      part = (int)w - row * a.splits;
      g0 = part * groups / a.splits;
      g1 = (part + 1) * groups / a.splits;
    }
    const int b = a.batch > 1 ? row / a.tokens : 0, t = row - b * a.tokens;
    Chunk<T, V> next[NS][2];
    auto load_group = [&](int g) {
      const bool is_q = g < gq;
      const RopeTensor& x = is_q ? a.q : a.k;
      // heads past the last: the last again, not stored
      const int h = min((g - (is_q ? 0 : gq)) * hpw + hl, x.heads - 1);
      const int64_t base = (int64_t)b * x.xb + (int64_t)t * x.xt + (int64_t)h * x.xh;
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const Slot<V, HALF> k(a, min(sl + 64 * i, slots - 1));
        next[i][0].load(x.x, base + k.ia);
        next[i][1].load(x.x, base + k.ib);
      }
    };
    load_group(g0);

    if constexpr (PACK) {
      for (int i = 0; i < 1 << lt; ++i) {
        const int at = (int)min((w << lt) + i, (int64_t)rows - 1);
        const int bi = a.batch > 1 ? at / a.tokens : 0;
        ang[wave].fill(a, a.pos + (int64_t)bi * a.pos_batch + (int64_t)(at - bi * a.tokens) * a.axes, lane, i * a.pairs);
      }
      ang[wave].filled();
    } else {
      ang[wave].compute(a, a.pos + (int64_t)b * a.pos_batch + (int64_t)t * a.axes, lane);
    }
    float c[NS][V], s[NS][V];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int slot = sl + 64 * i;
      const Slot<V, HALF> k(a, slot);
      if (slot < slots && k.turns) ang[wave].template take<V, HALF>(k, slot, c[i], s[i], tk * a.pairs);
    }
    if (!weights_there) {
#pragma unroll
      for (int i = 0; i < WL; ++i) weights[threadIdx.x + i * 64 * kRopeWaves] = w_mine[i];
      lds_barrier();
      weights_there = true;
    }

#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const RopeTensor& x = z ? a.k : a.q;
      const int first = z ? gq : 0;                    // the tensor's first group
      const int lo = max(g0, first), hi = min(g1, z ? groups : gq);
      if (lo >= hi) continue;
      float wa[NS][V], wb[NS][V];
      if constexpr (NORM) {
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          const Slot<V, HALF> k(a, min(sl + 64 * i, slots - 1));
#pragma unroll
          for (int j = 0; j < V; ++j) {
            wa[i][j] = weights[z * kRopeMaxHeadDim + k.ia + j];
            wb[i][j] = weights[z * kRopeMaxHeadDim + k.ib + j];
          }
        }
      }
      for (int g = lo; g < hi; ++g) {
        float fa[NS][V], fb[NS][V];
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          next[i][0].values(fa[i]);
          next[i][1].values(fb[i]);
        }
        if (g + 1 < g1) load_group(g + 1);
        const int h = (g - first) * hpw + hl;
        if constexpr (NORM) {
          float sum = 0.0f;
#pragma unroll
          for (int i = 0; i < NS; ++i) {
            float part_sum = 0.0f;
#pragma unroll
            for (int j = 0; j < V; ++j)
              part_sum = __builtin_fmaf(fa[i][j], fa[i][j], __builtin_fmaf(fb[i][j], fb[i][j], part_sum));
            sum += sl + 64 * i < slots ? part_sum : 0.0f;
          }
          const float rstd = rsqrt_of(__builtin_fmaf(run_sum(sum, a.lg), inv_dim, a.eps));
#pragma unroll
          for (int i = 0; i < NS; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
              fa[i][j] = fa[i][j] * rstd * wa[i][j];
              fb[i][j] = fb[i][j] * rstd * wb[i][j];
            }
        }
        const int64_t base = (int64_t)b * x.yb + (int64_t)t * x.yt + (int64_t)h * x.yh;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          const int slot = sl + 64 * i;
          const Slot<V, HALF> k(a, slot);
          if (!live || slot >= slots || h >= x.heads) continue;
          if (k.turns) turn_slot<V, HALF>(fa[i], fb[i], c[i], s[i]);
          store_vals<T, V>(x.y, base + k.ia, fa[i]);
          store_vals<T, V>(x.y, base + k.ib, fb[i]);
        }
      }
    }
  }
}

// The norm over all heads of a token where one wave can hold q (or k) of a
// token: job 2 row + z is tensor z of token row, its lanes as in the head
// kernel, G groups of heads in registers between the sum of squares and the
// rotation.  No barrier, and every wave's loads are all in flight at once (2 x
// 4099 tokens of 40 + 40 heads of 128, bf16: 69 us, 4.9 TB/s).
template <typename T, int V, bool HALF, int G>
__global__ __launch_bounds__(64 * kRopeWaves) void rope_token_wave_kernel(RopeArgs a) {
  __shared__ WaveAngles ang[kRopeWaves];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int slots = a.dim / (2 * V);
  const int sl = lane & ((1 << a.lg) - 1), hl = lane >> a.lg, hpw = 64 >> a.lg;
  const int tensors = a.k.heads > 0 ? 2 : 1;
  const int64_t total = (int64_t)a.batch * a.tokens * tensors;
  for (int64_t w = (int64_t)blockIdx.x * kRopeWaves + wave; w < total; w += (int64_t)gridDim.x * kRopeWaves) {
    const int row = (int)(tensors > 1 ? w >> 1 : w);
    const RopeTensor& x = tensors > 1 && (w & 1) ? a.k : a.q;
    const int b = a.batch > 1 ? row / a.tokens : 0, t = row - b * a.tokens;
    const int32_t* pos = a.pos + (int64_t)b * a.pos_batch + (int64_t)t * a.axes;
    const Slot<V, HALF> k(a, min(sl, slots - 1));
    Chunk<T, V> raw[G][2];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      // heads past the last: the last again, neither summed nor stored
      const int64_t base = (int64_t)b * x.xb + (int64_t)t * x.xt + (int64_t)min(g * hpw + hl, x.heads - 1) * x.xh;
      raw[g][0].load(x.x, base + k.ia);
      raw[g][1].load(x.x, base + k.ib);
    }
    ang[wave].compute(a, pos, lane);
    float sum = 0.0f;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float fa[V], fb[V], part = 0.0f;
      raw[g][0].values(fa);
      raw[g][1].values(fb);
#pragma unroll
      for (int j = 0; j < V; ++j) part = __builtin_fmaf(fa[j], fa[j], __builtin_fmaf(fb[j], fb[j], part));
      sum += sl < slots && g * hpw + hl < x.heads ? part : 0.0f;
    }
    const float rstd = rsqrt_of(run_sum(sum, 6) / (float)(x.heads * a.dim) + a.eps);
    float c[V], s[V];
    if (sl < slots && k.turns) ang[wave].template take<V, HALF>(k, sl, c, s);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int h = g * hpw + hl;
      if (sl >= slots || h >= x.heads) continue;
      raw[g][0].keep();
      raw[g][1].keep();
      float fa[V], fb[V], wa[V], wb[V];
      raw[g][0].values(fa);
      raw[g][1].values(fb);
      load_weight<V>(x, a.w_f32, (int64_t)h * a.dim + k.ia, wa);
      load_weight<V>(x, a.w_f32, (int64_t)h * a.dim + k.ib, wb);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        fa[j] = fa[j] * rstd * wa[j];
        fb[j] = fb[j] * rstd * wb[j];
      }
      if (k.turns) turn_slot<V, HALF>(fa, fb, c, s);
      const int64_t base = (int64_t)b * x.yb + (int64_t)t * x.yt + (int64_t)h * x.yh;
      store_vals<T, V>(x.y, base + k.ia, fa);
      store_vals<T, V>(x.y, base + k.ib, fb);
    }
  }
}

// The norm over all heads of a token: a workgroup takes q (blockIdx.y = 0) or
// k of one token after another, its lanes the (head, slot) items in order, NH
// each; the sums of squares are joined through LDS in wave order, and the
// token's cosines and sines are computed once into LDS.  The weights of a
// lane's items stay in registers over the tokens, and the next token's values
// are loaded before the current one is finished.  Items past a lane's NH (more
// than 1024 slots) are read twice, the second time from the L2.  4096 tokens of
// 96 + 96 heads of 128, bf16: 100 us, 4.0 TB/s (a barrier per token).
constexpr int kRopeMaxWaves = 8;
template <typename T, int V, bool HALF, int NH>
__global__ __launch_bounds__(64 * kRopeMaxWaves) void rope_token_kernel(RopeArgs a) {
  __shared__ float cs[2][2][kRopeMaxHeadDim / 2];
  __shared__ float part[2][kRopeMaxWaves];
  const int tid = threadIdx.x, n = blockDim.x, lane = tid & 63, wave = tid >> 6, waves = n >> 6;
  const RopeTensor x = blockIdx.y ? a.k : a.q;
  const int slots = a.dim / (2 * V), items = x.heads * slots;
  const int64_t rows = (int64_t)a.batch * a.tokens;
  auto at = [&](bool out, int64_t row, int h) -> int64_t {
    const int b = a.batch > 1 ? (int)row / a.tokens : 0, t = (int)row - b * a.tokens;
    return out ? (int64_t)b * x.yb + (int64_t)t * x.yt + (int64_t)h * x.yh
               : (int64_t)b * x.xb + (int64_t)t * x.xt + (int64_t)h * x.xh;
  };
  int head[NH], slot_of[NH];                     // items past the last: head -1
  float wa[NH][V], wb[NH][V];
#pragma unroll
  for (int i = 0; i < NH; ++i) {
    const int item = tid + i * n;
    head[i] = item < items ? item / slots : -1;
    slot_of[i] = item % slots;
    if (head[i] < 0) continue;
    const Slot<V, HALF> k(a, slot_of[i]);
    load_weight<V>(x, a.w_f32, (int64_t)head[i] * a.dim + k.ia, wa[i]);
    load_weight<V>(x, a.w_f32, (int64_t)head[i] * a.dim + k.ib, wb[i]);
  }
  Chunk<T, V> next[NH][2];
  auto load_token = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < NH; ++i) {
      if (head[i] < 0) continue;
      const Slot<V, HALF> k(a, slot_of[i]);
      const int64_t base = at(false, row, head[i]);
      next[i][0].load(x.x, base + k.ia);
      next[i][1].load(x.x, base + k.ib);
    }
  };
  auto squares = [&](const float (&va)[V], const float (&vb)[V], float acc) {
#pragma unroll
    for (int j = 0; j < V; ++j) acc = __builtin_fmaf(va[j], va[j], __builtin_fmaf(vb[j], vb[j], acc));
    return acc;
  };
  if ((int64_t)blockIdx.x < rows) load_token(blockIdx.x);
  int buf = 0;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, buf ^= 1) {
    if (a.pairs > 0) {
      const int b = a.batch > 1 ? (int)row / a.tokens : 0, t = (int)row - b * a.tokens;
      const int32_t* pos = a.pos + (int64_t)b * a.pos_batch + (int64_t)t * a.axes;
      for (int p = tid; p < a.pairs; p += n) {
        float c, s;
        cos_sin_turns(pair_turns(a, pos, p), c, s);
        cs[buf][0][p] = c * a.amplitude;
        cs[buf][1][p] = s * a.signed_amplitude;
      }
    }
    float fa[NH][V], fb[NH][V];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NH; ++i) {
      if (head[i] < 0) continue;
      next[i][0].values(fa[i]);
      next[i][1].values(fb[i]);
      sum = squares(fa[i], fb[i], sum);
    }
    for (int item = tid + NH * n; item < items; item += n) {
      const int h = item / slots;
      const Slot<V, HALF> k(a, item - h * slots);
      Chunk<T, V> ca, cb;
      ca.load(x.x, at(false, row, h) + k.ia);
      cb.load(x.x, at(false, row, h) + k.ib);
      float va[V], vb[V];
      ca.values(va);
      cb.values(vb);
      sum = squares(va, vb, sum);
    }
    if (row + gridDim.x < rows) load_token(row + gridDim.x);
    sum = run_sum(sum, 6);
    if (lane == 0) part[buf][wave] = sum;
    lds_barrier();               // one per token: the next one writes the other cs and part
    float all = 0.0f;
    for (int i = 0; i < waves; ++i) all += part[buf][i];
    const float rstd = rsqrt_of(all / (float)(x.heads * a.dim) + a.eps);
    auto finish = [&](int h, int slot, float (&va)[V], float (&vb)[V], const float (&ua)[V], const float (&ub)[V]) {
      const Slot<V, HALF> k(a, slot);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        va[j] = va[j] * rstd * ua[j];
        vb[j] = vb[j] * rstd * ub[j];
      }
      if (k.turns) {
        float c[V], s[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int p = k.pair(slot, j);
          c[j] = cs[buf][0][p];
          s[j] = cs[buf][1][p];
        }
        turn_slot<V, HALF>(va, vb, c, s);
      }
      const int64_t base = at(true, row, h);
      store_vals<T, V>(x.y, base + k.ia, va);
      store_vals<T, V>(x.y, base + k.ib, vb);
    };
#pragma unroll
    for (int i = 0; i < NH; ++i)
      if (head[i] >= 0) finish(head[i], slot_of[i], fa[i], fb[i], wa[i], wb[i]);
    for (int item = tid + NH * n; item < items; item += n) {
      const int h = item / slots, slot = item - h * slots;
      const Slot<V, HALF> k(a, slot);
      Chunk<T, V> ca, cb;
      ca.load(x.x, at(false, row, h) + k.ia);
      cb.load(x.x, at(false, row, h) + k.ib);
      float va[V], vb[V], ua[V], ub[V];
      ca.values(va);
      cb.values(vb);
      load_weight<V>(x, a.w_f32, (int64_t)h * a.dim + k.ia, ua);
      load_weight<V>(x, a.w_f32, (int64_t)h * a.dim + k.ib, ub);
      finish(h, slot, va, vb, ua, ub);
    }
  }
}

template <typename T, int V, bool HALF>
hipError_t launch_v(RopeArgs a, int norm, int cus, hipStream_t stream) {
  const int slots = a.dim / (2 * V);
  const int64_t rows = (int64_t)a.batch * a.tokens;
  a.lg = 0;
  while ((1 << a.lg) < slots && a.lg < 6) ++a.lg;
  const int hpw = 64 >> a.lg;
  if (norm == DDG_NORM_TOKEN) {
    const int tensors = a.k.heads > 0 ? 2 : 1;
    const int most_heads = std::max(a.q.heads, a.k.heads);
    if constexpr (V > 1) {
      const int groups = (most_heads + hpw - 1) / hpw;
      const int64_t grid = std::min<int64_t>((rows * tensors + kRopeWaves - 1) / kRopeWaves, (int64_t)cus * 64);
      auto launch = [&](auto kernel) {
        kernel<<<dim3((unsigned)grid), dim3(64 * kRopeWaves), 0, stream>>>(a);
        return hipGetLastError();
      };
      if (groups <= 2) return launch(rope_token_wave_kernel<T, V, HALF, 2>);
      if (groups <= 5) return launch(rope_token_wave_kernel<T, V, HALF, 5>);
      if (groups <= 8) return launch(rope_token_wave_kernel<T, V, HALF, 8>);
    }
    // lanes in whole waves, the same number of items (one or two) for nearly
    // all of them; as many workgroups as are resident at once
    const int64_t items = (int64_t)most_heads * slots;
    const int64_t most = 64 * kRopeMaxWaves;
    const int64_t per = std::min<int64_t>((items + most - 1) / most, 2);
    const int lanes = (int)std::min<int64_t>(((items + per - 1) / per + 63) / 64 * 64, most);
    const int64_t grid = std::min<int64_t>(rows, (int64_t)cus * std::max(1, 16 * 64 / lanes / tensors));
    const dim3 blocks((unsigned)grid, (unsigned)tensors);
    if (per == 1)
      rope_token_kernel<T, V, HALF, 1><<<blocks, dim3((unsigned)lanes), 0, stream>>>(a);
    else
      rope_token_kernel<T, V, HALF, 2><<<blocks, dim3((unsigned)lanes), 0, stream>>>(a);
    return hipGetLastError();
  }
  const int groups = (a.q.heads + hpw - 1) / hpw + (a.k.heads + hpw - 1) / hpw;
  // a token's heads go to several waves while tokens alone leave waves idle
  const int64_t want = (int64_t)cus * 16;
  a.splits = (int)std::max<int64_t>(1, std::min<int64_t>(groups, want / rows));
  int64_t waves = rows * a.splits;
  a.lt = 0;
  if (V > 1) {
    const int most_heads = std::max(a.q.heads, a.k.heads);
    while (most_heads <= hpw >> (a.lt + 1) && a.pairs << (a.lt + 1) <= kRopeMaxHeadDim / 2 &&
           rows >> (a.lt + 1) >= (int64_t)cus * 8)
      ++a.lt;
    if (a.lt > 0) waves = (rows + (1 << a.lt) - 1) >> a.lt;
  }
  const int64_t grid = std::min<int64_t>((waves + kRopeWaves - 1) / kRopeWaves, (int64_t)cus * 64);
  auto launch = [&](auto kernel) {
    kernel<<<dim3((unsigned)grid), dim3(64 * kRopeWaves), 0, stream>>>(a);
    return hipGetLastError();
  };
  if constexpr (V > 1) {
    if (a.lt > 0)
      return norm == DDG_NORM_HEAD ? launch(rope_head_kernel<T, V, HALF, true, true>)
                                   : launch(rope_head_kernel<T, V, HALF, false, true>);
  }
  return norm == DDG_NORM_HEAD ? launch(rope_head_kernel<T, V, HALF, true, false>)
                               : launch(rope_head_kernel<T, V, HALF, false, false>);
}

template <typename T, int V>
hipError_t launch_layout(const RopeArgs& a, int norm, bool half, int cus, hipStream_t stream) {
  return half ? launch_v<T, V, true>(a, norm, cus, stream) : launch_v<T, V, false>(a, norm, cus, stream);
}

// Chunks of V values are aligned in every row of x, and split the head.
bool chunks_of(const RopeArgs& a, int es, int v) {
  if (a.dim % (2 * v) || a.pairs % v) return false;
  auto ok = [&](const RopeTensor& x) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(x.x) | reinterpret_cast<uintptr_t>(x.y);
    const int64_t st = x.xb | x.xt | x.xh | x.yb | x.yt | x.yh;
    return x.heads == 0 || (at % (uintptr_t)(v * es) == 0 && st % v == 0);
  };
  return ok(a.q) && ok(a.k);
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, int norm, bool half, bool f32, int cus, hipStream_t stream) {
  // the widest chunks that the head, the rotated part and the rows allow; two
  // values (an even number of pairs, as 36 rotated values of 72) while a head's
  // slots are the lanes of a wave at most (8192 tokens of 16 + 16 such heads 32
  // us, 83 with a wave per head)
  const bool two = a.dim <= 256;
  if (f32) {
    if (chunks_of(a, 4, 4)) return launch_layout<float, 4>(a, norm, half, cus, stream);
    if (two && chunks_of(a, 4, 2)) return launch_layout<float, 2>(a, norm, half, cus, stream);
    return launch_layout<float, 1>(a, norm, half, cus, stream);
  }
  if (chunks_of(a, 2, 8)) return launch_layout<__bf16, 8>(a, norm, half, cus, stream);
  if (chunks_of(a, 2, 4)) return launch_layout<__bf16, 4>(a, norm, half, cus, stream);
  if (two && chunks_of(a, 2, 2)) return launch_layout<__bf16, 2>(a, norm, half, cus, stream);
  return launch_layout<__bf16, 1>(a, norm, half, cus, stream);
}

}  // namespace ddg

// Host only.  Pair i of `rot` values turns freq_i = base^(-2i / rot) per
// position; the scalings for contexts `factor` times the original length:
//   linear  freq_i / factor (positions interpolated);
//   ntk     base * factor^(rot / (rot - 2)): the first pair keeps its
//           frequency, the last one gets freq / factor;
//   yarn    pairs that turn at least beta_fast times over the original length
//           keep their frequency, those under beta_slow turns are divided by
//           factor, with a linear ramp over the pair index between; amplitude
//           0.1 ln(factor) + 1.
extern "C" int ddg_rope_frequencies(int rot_dim, double base, int scaling, double factor, double original_length,
                                    double beta_fast, double beta_slow, double* freqs, double* amplitude) {
  if (scaling < DDG_ROPE_SCALE_NONE || scaling > DDG_ROPE_SCALE_YARN || !freqs || !amplitude) return DDG_ERR_ARG;
  if (rot_dim < 2 || rot_dim % 2 || rot_dim > DDG_ROPE_MAX_HEAD_DIM) return DDG_ERR_SHAPE;
  if (!(base > 1.0) || !std::isfinite(base)) return DDG_ERR_ARG;
  if (scaling != DDG_ROPE_SCALE_NONE && (!(factor >= 1.0) || !std::isfinite(factor))) return DDG_ERR_ARG;
  if (scaling == DDG_ROPE_SCALE_NTK && rot_dim < 4) return DDG_ERR_SHAPE;
  if (scaling == DDG_ROPE_SCALE_YARN &&
      (!(original_length >= 1.0) || !std::isfinite(original_length) || !(beta_slow > 0.0) ||
       !(beta_fast >= beta_slow) || !std::isfinite(beta_fast)))
    return DDG_ERR_ARG;
  const int pairs = rot_dim / 2;
  const double b = scaling == DDG_ROPE_SCALE_NTK ? base * std::pow(factor, rot_dim / (rot_dim - 2.0)) : base;
  double low = 0.0, high = 0.0;
  if (scaling == DDG_ROPE_SCALE_YARN) {
    // pair index whose wavelength fits `turns` times into the original length
    auto pair_of = [&](double turns) {
      return rot_dim * std::log(original_length / (turns * 2.0 * M_PI)) / (2.0 * std::log(base));
    };
    low = std::max(std::floor(pair_of(beta_fast)), 0.0);
    high = std::min(std::ceil(pair_of(beta_slow)), rot_dim - 1.0);
  }
  for (int i = 0; i < pairs; ++i) {
    const double f = std::pow(b, -2.0 * i / rot_dim);
    if (scaling == DDG_ROPE_SCALE_LINEAR) {
      freqs[i] = f / factor;
    } else if (scaling == DDG_ROPE_SCALE_YARN) {
      const double ramp = std::min(std::max((i - low) / std::max(high - low, 0.001), 0.0), 1.0);
      freqs[i] = f * (1.0 - ramp) + f / factor * ramp;
    } else {
      freqs[i] = f;
    }
  }
  *amplitude = scaling == DDG_ROPE_SCALE_YARN ? 0.1 * std::log(factor) + 1.0 : 1.0;
  return DDG_OK;
}
