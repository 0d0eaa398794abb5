// Group-limited top-k routing of given logits.
//
// Handbook news post (hub.geekagi.cn), "真正难在三个环节" item 2 (a bias for balance that only
// selects) and the quoted tweet (softmax, sigmoid, sqrt(softplus) scores); "Hugging Face 图解
// Mixture of Experts（MoE）原理、训练与推理权衡", section "什么是稀疏性？" (KeepTopK, gates).
//
// moe_route_grouped.  The E experts form G groups of n = E / G.  An expert's key is its logit,
// or score + bias in fp64; a group's value is its largest key, or the sum of its two largest
// scores (+ bias).  The kept groups are the `kept` largest values, and the k largest keys of
// their experts are selected (ties to the lower index, both times).
//
// What it costs.  A token reads 4E bytes once and writes 8k; the work is the E scores, the two
// selections and the k gates, so at hundreds of experts it is bound by instruction issue.
//   - One warp per token.  A group belongs to a team of 32 / G' lanes (G' = G rounded up to a
//     power of two), so a lane finds the two largest keys of its part and a few
//     shuffles finish the group.
//   - The selection runs on fp32 keys a with a known bound |a - key| <= delta.  The kept groups'
//     keys are spread evenly over the lanes through shared memory; the k-th largest of the 32
//     lane maxima is a lower bound of the k-th largest key, so everything below it (less
//     2 delta) is out.  What is left, about k to 2k experts, gets one lane each: its key in
//     fp64, and its rank by counting the larger ones.  No round per selected expert.
//   - Where the border between kept and dropped groups is closer than fp32 holds, the experts
//     that can be among the groups' two largest are evaluated in fp64 (softmax: and its sum, as
//     for two candidates within 2 delta).  Where that leaves more than 32 experts, or fewer than k
//     are unmasked, the warp does the token again in fp64 alone.
//   - Rows of whole 16-byte pieces come by bulk copies.  A row with an infinite logit takes the
//     fp64 path, so the scores need no clamp.
// So every selection is the fp64 one; the fp32 pass only discards what cannot be selected.  The gates
// are fp64 too, but for the softmax's denominator over all experts (without renormalising), which
// is the fp32 pass's sum: at most 64 + 5 additions, 2 steps an exponential and half a step of each
// difference.  Summed in fp64 it took 121 us by a polynomial and 147 by exp() where this takes 80
// (32768 tokens, 896 experts, groups by their largest key).
#include <float.h>

#include "common.cuh"
#include "f32x2.cuh"
#include "tc_prims.cuh"

namespace moe {
namespace {

constexpr int kGroupWarps = 8;
constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ float wmax(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}
__device__ __forceinline__ float wsum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
__device__ __forceinline__ double wsum_d(double v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
__device__ __forceinline__ double wmax_d(double v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmax(v, __shfl_xor_sync(kFull, v, o));
  return v;
}

// A logit as the routing takes it: NaN counts as masked (-inf; fmaxf drops a NaN), +inf as the
// largest float.
__device__ __forceinline__ float clean_logit(float l) { return fminf(fmaxf(l, -INFINITY), FLT_MAX); }

__device__ __forceinline__ double score64(double l, int score) {
  if (score == MOE_SCORE_SIGMOID) return 1.0 / (1.0 + exp(-l));
  return sqrt(fmax(l, 0.0) + log1p(exp(-fabs(l))));
}

// The units' own exponential (base 2), reciprocal and square root, subnormals flushed: each is
// within 2 steps of its result.
__device__ __forceinline__ float ex2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float sqrt_fast(float x) {
  float r;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
constexpr float kLog2e = 1.44269504f;

// fp32 scores of two logits for discarding; 0 at -inf.  The exponent l log2(e) is rounded, so the
// error grows with |l| (2 + 1.2 |l| steps), but for l < -1 the score itself falls faster: over a
// row the error stays below the largest score times 2e-6 + 2.4e-7 |l of the largest score|,
// as long as that score is far above the flushed subnormals.
template <int SCORE>
__device__ __forceinline__ float2 score32(float x, float y) {
  if (SCORE == MOE_SCORE_SIGMOID)
    return make_float2(rcp_fast(1.f + ex2_fast(x * -kLog2e)), rcp_fast(1.f + ex2_fast(y * -kLog2e)));
  const f32x2 e = pack2(ex2_fast(fabsf(x) * -kLog2e), ex2_fast(fabsf(y) * -kLog2e));
  const float2 s = unpack2(add2(log1p_unit(e), pack2(fmaxf(x, 0.f), fmaxf(y, 0.f))));
  return make_float2(sqrt_fast(s.x), sqrt_fast(s.y));
}

struct Pick {
  int idx;        // lane j < k: the j-th selected expert
  double m, z;    // softmax: largest unmasked logit and sum of exp(l - m), if they were asked for
  double s;       // sigmoid, sqrt(softplus): the selected expert's score
};

struct GroupArgs {
  const float* logits;
  const float* bias;
  int32_t* topk_idx;
  float* topk_gate;
  int T, E, k, G, n, kept, team, chunks, top2, renorm;
  float scale;
  int* err;
};

// The whole selection of one token in fp64, by the warp.  A lane keeps the keys of its part of its
// group (every team-th expert) in local memory and its best one at hand; k rounds of an arg-max
// over the lanes follow.  One token here holds up its warp for some 15 us; 32768 tokens of 896 experts
// that all come here take 1.3 to 1.45 ms in place of 98 us (a router at its zero start, or an infinite
// or NaN bias).
template <int SCORE>
__device__ __noinline__ Pick route_token_fp64(const GroupArgs& a, const float* __restrict__ l) {
  const int lane = threadIdx.x & 31;
  const int L = a.team, g = lane / L, tl = lane - g * L;
  const bool in_g = g < a.G;
  const int count = in_g && tl < a.n ? (a.n - tl + L - 1) / L : 0;   // at most 64
  const int e0 = g * a.n + tl;
  double key[64];
  Pick out;
  out.m = 0.0;
  out.z = 1.0;
  if (SCORE == MOE_SCORE_SOFTMAX) {
    double m = -INFINITY, z = 0.0;
    for (int i = 0; i < count; ++i) m = fmax(m, (double)clean_logit(__ldg(l + e0 + i * L)));
    m = wmax_d(m);
    if (m > -INFINITY) {
#pragma unroll 2
      for (int i = 0; i < count; ++i) z += exp((double)clean_logit(__ldg(l + e0 + i * L)) - m);
      z = wsum_d(z);
      out.m = m;
      out.z = z;
    }
  }
  // keys; the group's two largest values; the lane's best key (the first of equal ones)
  const bool scored = a.bias || a.top2;
  double v1 = -INFINITY, v2 = -INFINITY, bk = -INFINITY;
  int bi = -1;
#pragma unroll 2
  for (int i = 0; i < count; ++i) {
    const float lf = clean_logit(__ldg(l + e0 + i * L));
    double k = (double)lf, v = k;
    if (scored && lf > -INFINITY) {
      v = SCORE == MOE_SCORE_SOFTMAX ? exp(k - out.m) / out.z : score64(k, SCORE);
      if (a.bias) {
        v += (double)__ldg(a.bias + e0 + i * L);
        if (v != v) v = -INFINITY;
        k = v;
      }
    }
    if (!a.top2) v = k;
    key[i] = k;
    if (v > v1) { v2 = v1; v1 = v; } else if (v > v2) v2 = v;
    if (bi < 0 || k > bk) { bk = k; bi = i; }
  }
  for (int o = 1; o < L; o <<= 1) {
    const double c = __shfl_xor_sync(kFull, v1, o), d = __shfl_xor_sync(kFull, v2, o);
    v2 = fmax(fmin(v1, c), fmax(v2, d));
    v1 = fmax(v1, c);
  }
  const double worth = a.top2 && v2 > -INFINITY ? v1 + v2 : v1;
  int rank = 0;
  for (int o = 0; o < a.G; ++o) {
    const double c = __shfl_sync(kFull, worth, o * L);
    rank += c > worth || (c == worth && o < g);
  }
  if (rank >= a.kept) bi = -1;                             // not a kept group: nothing to give
  unsigned long long taken = 0;
  out.idx = 0;
  for (int j = 0; j < a.k; ++j) {
    double wk = bk;
    int we = bi < 0 ? 0x7fffffff : e0 + bi * L;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const double c = __shfl_xor_sync(kFull, wk, o);
      const int ce = __shfl_xor_sync(kFull, we, o);
      if (ce != 0x7fffffff && (we == 0x7fffffff || c > wk || (c == wk && ce < we))) { wk = c; we = ce; }
    }
    if (lane == j) out.idx = we;
    if (bi >= 0 && we == e0 + bi * L) {                    // the owner looks for its next best
      taken |= 1ull << bi;
      bi = -1;
      for (int i = 0; i < count; ++i)
        if (!((taken >> i) & 1ull) && (bi < 0 || key[i] > bk)) { bk = key[i]; bi = i; }
    }
  }
  out.s = 0.0;
  if (SCORE != MOE_SCORE_SOFTMAX && lane < a.k) {
    const float lf = clean_logit(__ldg(l + out.idx));
    if (lf > -INFINITY) out.s = score64((double)lf, SCORE);
  }
  return out;
}

// A row of keys in shared memory as a lane sees it: its part of its group, in `chunks` chunks of
// four (VEC: four neighbouring experts).
template <bool VEC>
struct Part {
  int base, n, L, tl, chunks;
  bool in_g;
  __device__ __forceinline__ int place(int i) const { return VEC ? 4 * (tl + L * (i >> 2)) + (i & 3) : tl + L * i; }
  __device__ __forceinline__ bool have(int i) const { return in_g && place(i) < n; }
  // chunk c of p (global or shared), `none` where it does not exist
  __device__ __forceinline__ void get(const float* p, int c, float (&f)[4], float none) const {
    if constexpr (VEC) {
      float4 q = make_float4(none, none, none, none);
      if (have(4 * c)) q = *reinterpret_cast<const float4*>(p + base + place(4 * c));
      f[0] = q.x; f[1] = q.y; f[2] = q.z; f[3] = q.w;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) f[k] = have(4 * c + k) ? p[base + place(4 * c + k)] : none;
    }
  }
  __device__ __forceinline__ void put(float* p, int c, const float (&f)[4]) const {
    if constexpr (VEC) {
      if (have(4 * c)) *reinterpret_cast<float4*>(p + base + place(4 * c)) = make_float4(f[0], f[1], f[2], f[3]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (have(4 * c + k)) p[base + place(4 * c + k)] = f[k];
    }
  }
};

// Floats as integers of the same order (-0 as +0; never 0), and back.
__device__ __forceinline__ unsigned ordered32(float v) {
  const unsigned u = __float_as_uint(v + 0.f);
  return u ^ ((unsigned)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_ordered32(unsigned o) {
  return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
// Doubles as integers of the same order (-0 as +0).
__device__ __forceinline__ unsigned long long ordered(double v) {
  const long long b = __double_as_longlong(v + 0.0);
  return (unsigned long long)b ^ ((unsigned long long)(b >> 63) | 0x8000000000000000ull);
}

// Rank among c keys, one a lane (-inf in the lanes from c on): how many are larger, and of equal
// ones the lower lane first.  The upper halves of the keys' integers decide, unless two lanes have
// the same one.  Eight lanes' keys at a time: what lies past c outranks none of the c.
__device__ __forceinline__ int rank_of(double key, int c) {
  const int lane = threadIdx.x & 31;
  const unsigned long long ok = ordered(key);
  const unsigned hi = (unsigned)(ok >> 32);
  const unsigned same = __match_any_sync(kFull, lane < c ? hi : 0u);   // a key's half is never 0
  int r = 0;
  if (__all_sync(kFull, lane >= c || same == 1u << lane)) {
    for (int j0 = 0; j0 < c; j0 += 8)
#pragma unroll
      for (int j = 0; j < 8; ++j) r += __shfl_sync(kFull, hi, j0 + j) > hi;
  } else {
    for (int j = 0; j < c; ++j) r += __shfl_sync(kFull, ok, j) > ok - (j < lane ? 1 : 0);
  }
  return r;
}

// Softmax: sum of exp(l - m) over a row's unmasked logits in fp64, by the warp.
__device__ __forceinline__ double exact_sum(const float* __restrict__ l, int E, float m) {
  double z = 0.0;
#pragma unroll 2
  for (int e = threadIdx.x & 31; e < E; e += 32) z += exp((double)clean_logit(__ldg(l + e)) - (double)m);
  return wsum_d(z);
}
// The ranks of c candidates (expert e in this lane) by softmax + bias in fp64.
__device__ __noinline__ int exact_softmax_order(const float* __restrict__ l, const float* __restrict__ bias, int E,
                                                float m, int e, int c) {
  const double z = exact_sum(l, E, m);
  double key = -INFINITY;
  if ((threadIdx.x & 31) < c) key = exp((double)clean_logit(__ldg(l + e)) - (double)m) / z + (double)__ldg(bias + e);
  return rank_of(key, c);
}

// The rank of this lane's group by exact values, when the fp32 ones are too close at the border.
// sure: +1 or -1 for a group that the fp32 values put above or below every group in question, 0 for
// those; only their experts whose fp32 key is at least th (the group's second largest, or its
// largest, less twice the error) are evaluated in fp64.  m: softmax's largest logit.
template <bool VEC, int SCORE>
__device__ __noinline__ int exact_rank(const GroupArgs& a, const Part<VEC>& part, const float* l, const float* row,
                                       float th, float m, int sure) {
  const int lane = threadIdx.x & 31;
  const int L = a.team, g = lane / L;
  const double z = SCORE == MOE_SCORE_SOFTMAX ? exact_sum(l, a.E, m) : 1.0;
  double v1 = -INFINITY, v2 = -INFINITY;
  for (int c = 0; c < part.chunks && sure == 0; ++c) {
    float key[4];
    part.get(row, c, key, -INFINITY);
    if (!a.bias) {                                         // the row holds logits, not scores
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float x = clean_logit(key[k]);
        const float s = SCORE == MOE_SCORE_SOFTMAX ? __expf(x - m) / (float)z : score32<SCORE>(x, x).x;
        key[k] = x > -INFINITY ? s : -INFINITY;
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (!(key[k] > -INFINITY && key[k] >= th)) continue;
      const int e = part.base + part.place(4 * c + k);
      const double x = (double)clean_logit(__ldg(l + e));
      double v = SCORE == MOE_SCORE_SOFTMAX ? exp(x - (double)m) / z : score64(x, SCORE);
      if (a.bias) v += (double)__ldg(a.bias + e);
      if (v > v1) { v2 = v1; v1 = v; } else if (v > v2) v2 = v;
    }
  }
  __syncwarp();
  for (int o = 1; o < L; o <<= 1) {
    const double c = __shfl_xor_sync(kFull, v1, o), d = __shfl_xor_sync(kFull, v2, o);
    v2 = fmax(fmin(v1, c), fmax(v2, d));
    v1 = fmax(v1, c);
  }
  double worth = a.top2 && v2 > -INFINITY ? v1 + v2 : v1;
  if (sure) worth = sure > 0 ? INFINITY : -INFINITY;
  int rank = 0;
  for (int o = 0; o < a.G; ++o) {
    const double c = __shfl_sync(kFull, worth, o * L);
    rank += c > worth || (c == worth && o < g);
  }
  return rank;
}

// The v-th largest (v from 1) of the 32 lanes' values: a bitonic sort, descending by lane.
__device__ __forceinline__ float kth_of_lanes(float v, int kth) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1) {
#pragma unroll
    for (int o = size >> 1; o; o >>= 1) {
      const float c = __shfl_xor_sync(kFull, v, o);
      const bool up = ((lane & size) == 0) == ((lane & o) == 0);   // this lane keeps the larger
      v = up ? fmaxf(v, c) : fminf(v, c);
    }
  }
  return __shfl_sync(kFull, v, kth - 1);
}

// VEC: groups of whole 16-byte pieces; a warp's row comes by one bulk copy, asked for as soon as the
// token before has its candidates.  The row stays in shared memory, where the keys replace the
// logits (a bias given), so that the kernel needs few registers, whatever n, and 32 warps hide its
// chains of shuffles and fp64.  32768 tokens, 896 experts in 16 groups, k = 16, by logit: 63 us, and
// 71 us with all groups kept (75 and 106 with the keys in registers and 24 warps).  The two best of
// sqrt(softplus) + bias, 4 groups kept: 98 us, at 0.7 of the issue rate (reading and the largest
// logit 26, scores 30, groups 8, candidates 19, their fp64 order and the gates 15); its bytes alone
// need 18.
template <bool VEC, int SCORE>
__global__ void __launch_bounds__(32 * kGroupWarps, 4)
route_group_kernel(const __grid_constant__ GroupArgs a) {
  extern __shared__ __align__(16) float gsm[];
  __shared__ __align__(8) uint64_t s_bar[kGroupWarps];
  __shared__ int s_abort;
  __shared__ int s_group[kGroupWarps][32];                 // the kept groups, ascending
  __shared__ int s_cand[kGroupWarps][32];
  __shared__ double s_score[kGroupWarps][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int E = a.E, n = a.n, k = a.k, L = a.team;
  const int shift = __ffs(L) - 1;                          // lanes to groups: L is a power of two
  const unsigned inv_n = ((1u << 20) + n - 1) / n;         // rounded up
  const int pool = a.kept * n;                             // experts of the kept groups
  float* row = gsm + (size_t)w * ((E + 3) / 4 * 4);
  volatile int* abort_flag = &s_abort;
  const uint32_t bar = smem_u32(&s_bar[w]);
  if (threadIdx.x == 0) s_abort = 0;
  if (VEC && lane == 0) {
    mbar_init(bar, 1);
    fence_mbar_init();
  }
  __syncthreads();
  const int g = lane >> shift, tl = lane & (L - 1);        // this lane's group, its place in the team
  const bool in_g = g < a.G;
  const Part<VEC> part{g * n, n, L, tl, a.chunks, in_g};
  const bool biased = a.bias != nullptr;
  const bool by_logit = !biased && !a.top2;                // fp32 keys are exact
  const bool need_z = SCORE == MOE_SCORE_SOFTMAX && (!by_logit || !a.renorm);
  float bmax = 0.f;                                        // largest |bias|: part of the bound
  bool odd = false;                                        // a NaN or infinite bias: every token in fp64
  if (biased)
    for (int e = lane; e < E; e += 32) {
      const float b = fabsf(__ldg(a.bias + e));
      bmax = fmaxf(bmax, b);
      odd |= !(b < INFINITY);
    }
  bmax = wmax(bmax);
  odd = __any_sync(kFull, odd);
  const long long nw = (long long)gridDim.x * warps;
  const long long first = (long long)blockIdx.x * warps + w;
  auto ask = [&](const float* src) {                       // lane 0: a row into the buffer
    mbar_expect_tx(bar, (uint32_t)E * 4);
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(row)),
                 "l"(src), "r"((uint32_t)E * 4), "r"(bar)
                 : "memory");
  };
  if (VEC && lane == 0 && first < a.T) ask(a.logits + first * E);
  uint32_t parity = 0;
  for (long long t = first; t < a.T; t += nw) {
    const float* l = a.logits + t * E;
    if constexpr (VEC) {
      const bool got = mbar_wait(bar, parity, abort_flag, a.err);
      if (!__all_sync(kFull, got)) {
        if (lane == 0) mbar_wait_drain(bar, parity, a.err);   // the copy lands before the block ends
        break;
      }
      parity ^= 1u;
    } else {
      __syncwarp();                                        // the previous token's row is read
      for (int e = lane; e < E; e += 32) row[e] = __ldg(l + e);
      __syncwarp();
    }
    // -------------------------------------------------- fp32 keys, the groups' two largest
    float m = -INFINITY, z = 0.f, delta = 0.f;
    bool top = false;                                      // an infinite logit
    if (need_z || !by_logit) {
#pragma unroll 4
      for (int c = 0; c < a.chunks; ++c) {
        float f[4];
        part.get(row, c, f, -INFINITY);
        m = fmaxf(fmaxf(fmaxf(f[0], f[1]), fmaxf(f[2], f[3])), m);   // drops NaNs
      }
      m = wmax(m);
      top = m == INFINITY;
      m = fminf(m, FLT_MAX);
    }
    const bool dead = need_z && !(m > -INFINITY);          // every expert masked
    if (need_z && !dead) {
#pragma unroll 2
      for (int c = 0; c < a.chunks; ++c) {
        float f[4];
        part.get(row, c, f, -INFINITY);
#pragma unroll
        for (int i = 0; i < 4; ++i) z += expf(clean_logit(f[i]) - m);
      }
      z = wsum(z);
    }
    bool slow = odd || (top && !by_logit);
    const float iz = need_z ? __fdividef(1.f, z) : 0.f;
    auto score_of = [&](float x, float y) {
      if (SCORE == MOE_SCORE_SOFTMAX) return make_float2(__expf(x - m) * iz, __expf(y - m) * iz);
      return score32<SCORE>(x, y);
    };
    float g1 = -INFINITY, g2 = -INFINITY;
    if (by_logit) {
      if (a.kept < a.G) {
#pragma unroll 4
        for (int c = 0; c < a.chunks; ++c) {
          float f[4];
          part.get(row, c, f, -INFINITY);
          g1 = fmaxf(fmaxf(fmaxf(f[0], f[1]), fmaxf(f[2], f[3])), g1);
        }
        g1 = fminf(g1, FLT_MAX);
      }
    } else {
#pragma unroll 2
      for (int c = 0; c < a.chunks; ++c) {
        float f[4], b[4] = {0.f, 0.f, 0.f, 0.f};
        part.get(row, c, f, -INFINITY);
        if (biased) part.get(a.bias, c, b, 0.f);
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const float x = f[i], y = f[i + 1];
          const float2 s = score_of(x, y);
          const float2 key = unpack2(add2(pack2(s.x, s.y), pack2(b[i], b[i + 1])));
          f[i] = x > -INFINITY ? key.x : -INFINITY;
          f[i + 1] = y > -INFINITY ? key.y : -INFINITY;
          const float hi = fmaxf(f[i], f[i + 1]), lo = fminf(f[i], f[i + 1]);
          g2 = fmaxf(fmaxf(g2, lo), fminf(g1, hi));
          g1 = fmaxf(g1, hi);
        }
        if (biased) part.put(row, c, f);
      }
      // the scores' error relative to the largest one, the largest logit's (see score32; softmax:
      // the sum and its reciprocal instead), and one rounding of s + b
      const float smax = dead ? 0.f : score_of(m, m).x;
      const float rel = SCORE == MOE_SCORE_SOFTMAX ? 3e-6f : 2e-6f + 2.4e-7f * fmaxf(0.f, -m);
      delta = rel * smax + 2.4e-7f * bmax;
      slow |= !(smax > 1e-12f);                            // near the flushed subnormals
    }
    // -------------------------------------------------- groups
    bool keep = in_g;
    if (a.kept < a.G) {
      for (int o = 1; o < L; o <<= 1) {
        const float c1 = __shfl_xor_sync(kFull, g1, o), c2 = __shfl_xor_sync(kFull, g2, o);
        g2 = fmaxf(fminf(g1, c1), fmaxf(g2, c2));
        g1 = fmaxf(g1, c1);
      }
      // the kept groups, one warp maximum each: a value as an integer of its order, of equal ones
      // the lower group
      const float gv = a.top2 && g2 > -INFINITY ? g1 + g2 : g1;
      unsigned left = in_g ? ordered32(gv) : 0u, worst = 0u;   // no value's integer is 0
      keep = false;
      for (int j = 0; j < a.kept; ++j) {
        worst = __reduce_max_sync(kFull, left);
        const int best_g = (__ffs(__ballot_sync(kFull, left == worst)) - 1) >> shift;
        if (g == best_g) {
          keep = true;
          left = 0u;
        }
      }
      if (!by_logit) {                                     // the border must be wider than the error
        const float lo = from_ordered32(worst), hi = from_ordered32(__reduce_max_sync(kFull, left));
        const float wide = 6.f * delta + 2.4e-7f * (fabsf(lo) + fabsf(hi));   // more than two values' errors
        if (!(lo - hi > wide) && hi > -INFINITY) {
          // above every dropped value by more than that: kept for certain; below every kept one: dropped
          const int sure = gv - hi > wide ? 1 : lo - gv > wide ? -1 : 0;
          keep = exact_rank<VEC, SCORE>(a, part, l, row, (a.top2 ? g2 : g1) - 2.f * delta, m, sure) < a.kept && in_g;
        }
      }
    }
    const unsigned heads = __ballot_sync(kFull, keep && tl == 0);
    if (keep && tl == 0) s_group[w][__popc(heads & ((1u << lane) - 1u))] = g;
    if (!biased) delta = 0.f;                              // experts by logit, whatever the groups go by
    __syncwarp();                                          // the keys and the groups are written
    // -------------------------------------------------- candidates
    // expert number p of the kept groups (p / n by a product: with p < 1024 and an excess of inv_n n
    // over 2^20 below n <= 1024, the quotient's excess stays below 1 / n)
    auto expert = [&](int p) {
      if (a.kept == a.G) return p;
      const int o = (int)((unsigned)p * inv_n >> 20);
      return s_group[w][o] * n + (p - o * n);
    };
    float best = -INFINITY;
#pragma unroll 1
    for (int p = lane; p < pool; p += 32) best = fmaxf(best, row[expert(p)]);
    best = fminf(best, FLT_MAX);
    float tau = kth_of_lanes(best, k);
    // the keys not below the threshold, in index order; the first 32 get a lane each
    auto compact = [&]() {
      const float th = tau - 2.f * delta - (delta > 0.f ? 2.4e-7f * fabsf(tau) : 0.f);
      int c = 0;
#pragma unroll 1
      for (int p0 = 0; p0 < pool; p0 += 32) {
        const int p = p0 + lane;
        const int e = p < pool ? expert(p) : 0;
        const bool in = p < pool && row[e] >= th;
        const unsigned b = __ballot_sync(kFull, in);
        const int at = c + __popc(b & ((1u << lane) - 1u));
        if (in && at < 32) s_cand[w][at] = e;
        c += __popc(b);
      }
      return c;
    };
    int c = compact();
    if (c > 32 && tau > -INFINITY) {
      // the lane maxima bound it too loosely (many selected, or unlucky): halve the way from
      // the bound to the largest key, keeping at least k keys above it
      float lo = tau, hi = wmax(best);
      for (int it = 0; it < 24; ++it) {
        const float mid = 0.5f * lo + 0.5f * hi;
        int above = 0;
        for (int p = lane; p < pool; p += 32) above += row[expert(p)] >= mid;
        above = (int)__reduce_add_sync(kFull, (unsigned)above);
        if (above >= k) lo = mid; else hi = mid;
        if (above >= k && above <= 32) break;
      }
      tau = lo;
      __syncwarp();
      c = compact();
    }
    __syncwarp();
    slow = slow || !(tau > -INFINITY) || c > 32 || c < k;
    int e = 0;
    float af = 0.f;
    if (lane < c && lane < 32) {
      e = s_cand[w][lane];
      af = row[e];
    }
    if (VEC && biased) fence_proxy_async_smem();           // the keys were written before the copy writes there
    __syncwarp();                                          // the row is done with
    if (VEC && lane == 0 && t + nw < a.T) ask(l + nw * E);
    // -------------------------------------------------- exact order of what is left
    Pick pick;
    pick.idx = 0;
    pick.m = (double)m;
    pick.z = (double)z;
    pick.s = 0.0;
    if (!slow) {
      double key = -INFINITY, s = 0.0;
      if (lane < c) {
        if (SCORE == MOE_SCORE_SOFTMAX && biased) {
          key = (double)af;
        } else {
          key = (double)clean_logit(biased ? __ldg(l + e) : af);
          if (SCORE != MOE_SCORE_SOFTMAX) s = score64(key, SCORE);
          if (biased) key = s + (double)__ldg(a.bias + e);
        }
      }
      int r = rank_of(key, c);
      if (SCORE == MOE_SCORE_SOFTMAX && biased) {
        // these keys are fp32: where two are within their error, fp64 decides
        bool near = false;
        for (int j = 0; j < c; ++j) {
          const float o = __shfl_sync(kFull, af, j);       // by every lane, whatever it has found
          near |= fabsf(o - af) <= 2.f * delta && j != lane;
        }
        if (__any_sync(kFull, near && lane < c)) r = exact_softmax_order(l, a.bias, E, m, e, c);
      }
      if (lane < c && r < k) {                             // every lane has read its candidate
        s_cand[w][r] = e;
        s_score[w][r] = s;
      }
      __syncwarp();
      if (lane < k) {
        pick.idx = s_cand[w][lane];
        pick.s = s_score[w][lane];
      }
    }
    if (slow) pick = route_token_fp64<SCORE>(a, l);
    // -------------------------------------------------- gates (fp64, rounded once; pick.z: see above)
    double s = 0.0;
    if (SCORE == MOE_SCORE_SOFTMAX) {
      const float lf = lane < k ? clean_logit(__ldg(l + pick.idx)) : -INFINITY;
      const double mm = a.renorm ? (double)wmax(lf) : pick.m;
      if (lf > -INFINITY) s = exp((double)lf - mm);
      if (!a.renorm) s /= pick.z;
    } else if (lane < k) {
      s = pick.s;
    }
    if (a.renorm) {
      const double tot = wsum_d(s);
      s = tot > 0.0 ? s / tot : 0.0;
    }
    if (lane < k) {
      a.topk_idx[t * k + lane] = pick.idx;
      a.topk_gate[t * k + lane] = (float)(s * (double)a.scale);
    }
    __syncwarp();                                          // the candidates' lists are read
  }
}

// Warps a block: eight, or fewer where the tokens would leave multiprocessors without any.
template <bool VEC, int SCORE>
moe_status run_group(const GroupArgs& a, cudaStream_t s) {
  const int sms = num_sms();
  int warps = (a.T + sms - 1) / sms;
  if (warps > kGroupWarps) warps = kGroupWarps;
  const size_t smem = (size_t)warps * ((a.E + 3) / 4 * 4) * sizeof(float);   // at most 32 KB
  long long blocks = ((long long)a.T + warps - 1) / warps;
  const long long cap = (long long)sms * 4;
  if (blocks > cap) blocks = cap;
  route_group_kernel<VEC, SCORE><<<(unsigned)blocks, 32 * warps, smem, s>>>(a);
  return check_launch();
}

}  // namespace

moe_status launch_route_grouped(const float* logits, int T, int E, int k, int n_groups, int groups_kept,
                                int group_score, int score, int renorm, float scale, const float* bias,
                                int32_t* topk_idx, float* topk_gate, cudaStream_t s) {
  GroupArgs a{logits, bias, topk_idx, topk_gate, T, E, k, n_groups, E / n_groups, groups_kept, 0, 0,
              group_score == MOE_GROUP_TOP2, renorm, scale, err_ptr()};
  int p2 = 1;
  while (p2 < n_groups) p2 <<= 1;
  a.team = 32 / p2;
  const bool vec = a.n % 4 == 0 && aligned16(logits) && aligned16(bias);
  a.chunks = (a.n + 4 * a.team - 1) / (4 * a.team);
  if (score == MOE_SCORE_SOFTMAX)
    return vec ? run_group<true, MOE_SCORE_SOFTMAX>(a, s) : run_group<false, MOE_SCORE_SOFTMAX>(a, s);
  if (score == MOE_SCORE_SIGMOID)
    return vec ? run_group<true, MOE_SCORE_SIGMOID>(a, s) : run_group<false, MOE_SCORE_SIGMOID>(a, s);
  return vec ? run_group<true, MOE_SCORE_SQRT_SOFTPLUS>(a, s) : run_group<false, MOE_SCORE_SQRT_SOFTPLUS>(a, s);
}

}  // namespace moe
