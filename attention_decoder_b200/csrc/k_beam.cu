// Beam selection: the best n_out of n_beams x vocab continuations of each group.
//
// A candidate (beam b, token v) scores s_b + x_bv - log sum_v exp x_bv. Within a row the order is that of the logits, so
// a block needs only its part's n_out largest logits, its maximum and its sum of exponentials: one pass over the
// logits (k_beam_parts), which bounds the work at 4 bytes a logit. A block per group then merges the parts
// (k_beam_merge): the log-sum-exps and the scores in 64 bits, so that candidates of different beams are ordered as in
// exact arithmetic down to the 2^-22 of the exponentials; ties go to the lowest (beam, token).
// Latency bounds both: 4 beams of 128000 tokens 8.9 us for 2 MB, 12 x 5 beams of 50001 18.8 us for 12 MB, half in each kernel.
#include <math_constants.h>

#include "kernels.cuh"

namespace lfm3 {

constexpr int BM_THREADS = 256;
constexpr int BM_WARPS = BM_THREADS / 32;
constexpr int BM_CAP = 256;  // candidates of a part above its threshold that are ranked directly

// Order-preserving map of finite floats and infinities to unsigned (NaN is mapped by the callers). Zeros of either sign are one
// value: -0 + 0 is +0.
DEVI uint32_t ord_f(float x) {
  const uint32_t u = __float_as_uint(__fadd_rn(x, 0.f));
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
DEVI float unord_f(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }
DEVI float ex2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr uint32_t ORD_NEG_INF = 0x007fffffu;  // ord_f(-inf)

// Part c of row r: granules (16-byte groups of the row, counted from the 16-byte boundary at or below its start)
// [c * 256 * IT, ...). Every thread keeps IT granules in registers. With full warps of 32 threads that all hold a valid
// logit, the q-th largest thread maximum of each of n such warps is exceeded or met by q of its logits, so with q n >= K
// the smallest of them is a threshold that at least K logits of the part reach: usually little more than K do, and those
// are ranked all against all. (A part where more than BM_CAP do finds the K-th largest (logit, -index) bit by bit.)
template <int IT>
__global__ void __launch_bounds__(BM_THREADS) k_beam_parts(const float* __restrict__ logits, long long ld, int V, int K,
                                                           const float* __restrict__ scores, const int* __restrict__ done,
                                                           float2* __restrict__ stats, int2* __restrict__ lists) {
  __shared__ uint64_t cand[BM_CAP];
  __shared__ float vals[4 * IT * BM_THREADS];
  __shared__ uint32_t wmax[BM_WARPS], wthr[BM_WARPS];
  __shared__ float wsum[BM_WARPS];
  __shared__ int cnt[2];
  const int part = blockIdx.x, row = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  pdl_launch_dependents();
  // a row that does not count (finished, or without a score) is read all the same, so that its logits need not wait for this
  const bool unused = (done && __ldcg(done + row)) || !(__ldcg(scores + row) > -CUDART_INF_F);
  const float* x = logits + (size_t)row * ld;
  const int shift = (int)((reinterpret_cast<uintptr_t>(x) & 15) >> 2);  // logits of the first granule before the row
  const float4* g0 = reinterpret_cast<const float4*>(x - shift);
  const int G = (V + shift + 3) / 4, first = part * BM_THREADS * IT;
  float v[4 * IT];
  if (4 * first >= shift && 4 * (first + BM_THREADS * IT) - shift <= V) {
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const float4 t = __ldcg(g0 + first + i * BM_THREADS + tid);
      v[4 * i] = t.x; v[4 * i + 1] = t.y; v[4 * i + 2] = t.z; v[4 * i + 3] = t.w;
    }
  } else {  // a part with an end of the row
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int g = first + i * BM_THREADS + tid, e = 4 * g - shift;  // e: index of the granule's first logit
#pragma unroll
      for (int k = 0; k < 4; ++k) v[4 * i + k] = g < G && e + k >= 0 && e + k < V ? __ldcg(x + e + k) : -CUDART_INF_F;
    }
  }
  if (unused) return;
  if (tid < 2) cnt[tid] = 0;
  float big = -CUDART_INF_F;  // the thread's largest logit (a NaN counts as none)
#pragma unroll
  for (int k = 0; k < 4 * IT; ++k) big = fmaxf(big, v[k]);
  const uint32_t tm = ord_f(big);
  const int nfull = min(BM_WARPS, (G - first) / 32);
  const int q = nfull > 0 ? (K + nfull - 1) / nfull : 33;
  uint32_t cur = tm, t = 0;
  for (int i = 0; i < min(q, 32); ++i) {  // the warp's q-th largest thread maximum
    t = __reduce_max_sync(0xffffffffu, cur);
    if (i == 0 && lane == 0) wmax[warp] = t;
    if (lane == __ffs(__ballot_sync(0xffffffffu, cur == t)) - 1) cur = 0;
  }
  if (lane == 0) wthr[warp] = q <= 32 && warp < nfull ? t : q <= 32 ? 0xffffffffu : 0u;
  __syncthreads();
  uint32_t mk = 0, thr = 0xffffffffu;
#pragma unroll
  for (int w = 0; w < BM_WARPS; ++w) {
    mk = max(mk, wmax[w]);
    thr = min(thr, wthr[w]);
  }
  thr = max(thr, ORD_NEG_INF + 1);  // -inf is no candidate
  const float m = unord_f(mk);
  float s = 0.f;
  if (mk > ORD_NEG_INF) {
#pragma unroll
    for (int k = 0; k < 4 * IT; ++k) s += ex2_ftz((v[k] - m) * 1.4426950408889634f);
  } else {  // nothing above -inf: a NaN, which no maximum shows, still has to reach the row's sum
#pragma unroll
    for (int k = 0; k < 4 * IT; ++k) s = v[k] != v[k] ? v[k] : s;
  }
  s = warp_sum(s);
  if (lane == 0) wsum[warp] = s;
  const float floor_ = unord_f(thr);
#pragma unroll
  for (int k = 0; k < 4 * IT; ++k)
    if (v[k] >= floor_) {
      const int at = atomicAdd(&cnt[0], 1);
      const int idx = 4 * (first + (k >> 2) * BM_THREADS + tid) - shift + (k & 3);
      if (at < BM_CAP) cand[at] = ((uint64_t)ord_f(v[k]) << 32) | (0xffffffffu - (uint32_t)idx);
    }
  __syncthreads();
  int n = cnt[0];
  if (n > BM_CAP) {  // the K-th largest key (keys are distinct), from its highest bit down; rare, so out of the registers
#pragma unroll
    for (int k = 0; k < 4 * IT; ++k) vals[k * BM_THREADS + tid] = v[k];
    __syncwarp();
    auto key_at = [&](int k) -> uint64_t {
      const float f = vals[k * BM_THREADS + tid];
      const int idx = 4 * (first + (k >> 2) * BM_THREADS + tid) - shift + (k & 3);
      return ((uint64_t)(f == f ? ord_f(f) : ORD_NEG_INF) << 32) | (0xffffffffu - (uint32_t)idx);
    };
    uint64_t lo = 0;
#pragma unroll 1
    for (int bit = 63; bit >= 0; --bit) {
      const uint64_t c = lo | (1ull << bit);
      int mine = 0;
#pragma unroll 1
      for (int k = 0; k < 4 * IT; ++k) mine += key_at(k) >= c;
      mine = __reduce_add_sync(0xffffffffu, mine);
      __syncthreads();
      if (tid == 0) cnt[1] = 0;
      __syncthreads();
      if (lane == 0) atomicAdd(&cnt[1], mine);
      __syncthreads();
      if (cnt[1] >= K) lo = c;
    }
    __syncthreads();
    if (tid == 0) cnt[0] = 0;
    __syncthreads();
#pragma unroll 1
    for (int k = 0; k < 4 * IT; ++k)
      if (key_at(k) >= lo) cand[atomicAdd(&cnt[0], 1)] = key_at(k);
    __syncthreads();
    n = cnt[0];
  }
  const size_t at = (size_t)row * gridDim.x + part;
  int2* list = lists + at * K;
  for (int i0 = 0; i0 < n; i0 += BM_THREADS / 8) {  // eight lanes a candidate
    const int i = i0 + (tid >> 3);
    const uint64_t mine = i < n ? cand[i] : 0;
    int rank = 0;
#pragma unroll 4
    for (int j = tid & 7; j < n; j += 8) rank += cand[j] > mine;
#pragma unroll
    for (int d = 4; d; d >>= 1) rank += __shfl_xor_sync(0xffffffffu, rank, d);
    if (i < n && (tid & 7) == 0 && rank < K)
      list[rank] = make_int2(__float_as_int(unord_f((uint32_t)(mine >> 32))), (int)(0xffffffffu - (uint32_t)mine));
  }
  for (int i = n + tid; i < K; i += BM_THREADS) list[i] = make_int2(__float_as_int(-CUDART_INF_F), -1);
  if (tid == 0) {
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < BM_WARPS; ++w) sum += wsum[w];
    stats[at] = make_float2(m, sum);
  }
}

struct BeamBest {
  double score;
  int idx, list;  // idx: beam * V + token; list: where it comes from (-1: none)
};
DEVI bool better(const BeamBest& a, const BeamBest& b) {
  return a.list >= 0 && (b.list < 0 || a.score > b.score || (a.score == b.score && a.idx < b.idx));
}
DEVI BeamBest shfl_best(BeamBest b, int o) {
  b.score = __shfl_xor_sync(0xffffffffu, b.score, o);
  b.idx = __shfl_xor_sync(0xffffffffu, b.idx, o);
  b.list = __shfl_xor_sync(0xffffffffu, b.list, o);
  return b;
}

// One block per group over the n_beams x parts sorted lists, dealt to the warps in turn (so that each sees every beam). As in a
// part, the smallest of the warps' q-th largest list heads, q times the warps >= K, is a threshold that at least K entries
// reach (scores compared as fp32 rounded down, which keeps the order), and so is the smallest of their largest eighth entries;
// a thread takes its lists' entries while they reach it,
// eight of them at a time. More than BM_RANK_CAP (few lists, or beams far apart) are cut down by a better bound, sought bit by
// bit; what is left is ranked all against all. Ties can leave too many all the same: then the lists merge head by head.
constexpr int BM_MTHREADS = 512, BM_MWARPS = BM_MTHREADS / 32, BM_MERGE_CAP = 2048, BM_RANK_CAP = 512;

// Order-preserving map of doubles (no NaN; zeros as in ord_f).
DEVI uint64_t ord_d(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(__dadd_rn(x, 0.0));
  return u >> 63 ? ~u : u | (1ull << 63);
}
DEVI double unord_d(uint64_t k) { return __longlong_as_double((long long)(k >> 63 ? k & ~(1ull << 63) : ~k)); }

__global__ void __launch_bounds__(BM_MTHREADS) k_beam_merge(int B, int V, int K, int parts, const float* __restrict__ scores,
                                                           const int* __restrict__ done, int end_token,
                                                           const float2* __restrict__ stats, const int2* __restrict__ lists,
                                                           float* __restrict__ out_score, int* __restrict__ out_parent,
                                                           int* __restrict__ out_token) {
  extern __shared__ unsigned char taken[];  // head-by-head merge: entries taken from list l
  __shared__ double off[BEAM_MAX_BEAMS];    // s_b - log sum_v exp(x_bv - top_b); of a finished beam s_b; NaN: no candidates
  __shared__ float top[BEAM_MAX_BEAMS];     // the row's maximum: subtracted first, whatever its size
  __shared__ int live[BEAM_MAX_BEAMS];      // beams with lists of candidates
  __shared__ bool fin[BEAM_MAX_BEAMS];
  __shared__ uint64_t cs[BM_MERGE_CAP];
  __shared__ int ci[BM_MERGE_CAP];
  __shared__ unsigned short sel[BM_RANK_CAP];
  __shared__ uint32_t wthr[2 * BM_MWARPS];
  __shared__ BeamBest wbest[BM_MWARPS];
  __shared__ int nlive, cnt, nsel;
  const int grp = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, row0 = grp * B;
  if (tid == 0) nlive = cnt = nsel = 0;
  pdl_wait();
  pdl_launch_dependents();
  __syncthreads();
  for (int b = warp; b < B; b += BM_MWARPS) {
    const float sb = __ldcg(scores + row0 + b);
    const bool f = done && __ldcg(done + row0 + b);
    const float2* st = stats + (size_t)(row0 + b) * parts;
    double o = CUDART_NAN;
    float M = -CUDART_INF_F;
    if (!f && sb > -CUDART_INF_F) {
      const float2 none = make_float2(-CUDART_INF_F, 0.f), first = lane < parts ? __ldcg(&st[lane]) : none;
      M = first.x;
      for (int p = lane + 32; p < parts; p += 32) M = fmaxf(M, __ldcg(&st[p]).x);
      M = warp_max(M);
      double S = 0.0;
      for (int p = lane; p < parts; p += 32) {
        const float2 a = p == lane ? first : __ldcg(&st[p]);
        S += (double)(a.y * (a.x == -CUDART_INF_F ? 0.f : ex2_ftz((a.x - M) * 1.4426950408889634f)));
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) S += __shfl_xor_sync(0xffffffffu, S, d);
      // S: NaN with a NaN or +inf in the row, 0 if all are -inf. Its logarithm from an exponent and an fp32 logarithm of a
      // value in [1, 2), which is off by less than 2^-24
      if (S > 0.0) {
        const long long u = __double_as_longlong(S);
        const int ex = (int)(u >> 52) - 1023;
        const float ma = (float)__longlong_as_double((u & 0xFFFFFFFFFFFFFll) | 0x3FF0000000000000ll);
        o = (double)sb - ((double)ex * 0.6931471805599453 + (double)logf(ma));
      }
    } else if (f && sb > -CUDART_INF_F) {
      o = (double)sb;
    }
    if (lane == 0) {
      off[b] = o;
      top[b] = M;
      fin[b] = f;
      if (o == o) {
        if (f) {
          const int at = atomicAdd(&cnt, 1);
          cs[at] = ord_d(o);
          ci[at] = b * V + end_token;
        } else {
          live[atomicAdd(&nlive, 1)] = b;
        }
      }
    }
  }
  __syncthreads();
  const int H = nlive * parts;
  auto score_of = [&](int b, float x) -> double { return off[b] + ((double)x - (double)top[b]); };
  auto list_of = [&](int beam, int p) -> const int2* { return lists + ((size_t)(row0 + beam) * parts + p) * K; };
  auto take = [&](int b, int token, double sc) {
    const int at = atomicAdd(&cnt, 1);
    if (at < BM_MERGE_CAP) {
      cs[at] = ord_d(sc);
      ci[at] = b * V + token;
    }
  };
  auto bound_of = [&](int b, float x, double& sc) -> uint32_t {  // the score, rounded down to fp32
    sc = score_of(b, x);
    return x > -CUDART_INF_F ? ord_f(__double2float_rd(sc)) : 0u;
  };
  const int q = (K + BM_MWARPS - 1) / BM_MWARPS, deal = BM_MWARPS * lane + warp;  // lists deal, deal + BM_MTHREADS, ..
  const int2 none = make_int2(__float_as_int(-CUDART_INF_F), 0);
  int2 e[8];  // eight entries of a list
  auto load = [&](const int2* list, int i0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = i0 + i < K ? __ldcg(list + i0 + i) : none;
  };
  int b = 0;
  const int2* list = nullptr;
  auto go = [&](int l) {
    const int j = l / parts;
    b = live[j];
    list = list_of(b, l - j * parts);
  };
  uint32_t tm = 0, thr = 0;
  double sc;
  for (int l = deal + (H - 1 - deal) / BM_MTHREADS * BM_MTHREADS; l >= deal && deal < H; l -= BM_MTHREADS) {
    go(l);
    if (l == deal)
      load(list, 0);  // the thread's first list stays in registers
    else
      e[0] = __ldcg(list);
    tm = max(tm, bound_of(b, __int_as_float(e[0].x), sc));
  }
  // two bounds: the warps' q-th largest heads, and the largest eighth entries (eight for each warp: more than any K)
  static_assert(8 * BM_MWARPS >= BEAM_MAX_OUT, "eight entries a warp are enough");
  const uint32_t t8 = __reduce_max_sync(0xffffffffu, deal < H ? bound_of(b, __int_as_float(e[7].x), sc) : 0u);
  uint32_t t = 0;
  for (int i = 0; i < q; ++i) {  // the warp's q-th largest thread maximum (0 if there are fewer lists)
    t = __reduce_max_sync(0xffffffffu, tm);
    if (lane == __ffs(__ballot_sync(0xffffffffu, tm == t)) - 1) tm = 0;
  }
  if (lane == 0) {
    wthr[warp] = t;
    wthr[BM_MWARPS + warp] = t8;
  }
  __syncthreads();
  uint32_t thr8 = 0xffffffffu;
  thr = 0xffffffffu;
#pragma unroll
  for (int w = 0; w < BM_MWARPS; ++w) {
    thr = min(thr, wthr[w]);
    thr8 = min(thr8, wthr[BM_MWARPS + w]);
  }
  thr = max(thr, thr8);
  __syncthreads();
  for (int l = deal; l < H; l += BM_MTHREADS) {
    if (l != deal) {
      go(l);
      load(list, 0);
    }
    bool more = true;
    for (int i0 = 0; more && i0 < K; i0 += 8) {
      if (i0) load(list, i0);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (!more) break;
        const uint32_t k = bound_of(b, __int_as_float(e[i].x), sc);
        more = k != 0 && k >= thr;
        if (more) take(b, e[i].y, sc);
      }
    }
  }
  __syncthreads();
  int n = cnt;
  const bool many = n > BM_RANK_CAP;
  if (many && n <= BM_MERGE_CAP) {
    uint32_t lo = 0;  // a bound on the scores' upper halves that K candidates reach
#pragma unroll 1
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t c = lo | (1u << bit);
      int reach = 0;
      for (int i = tid; i < n; i += BM_MTHREADS) reach += (uint32_t)(cs[i] >> 32) >= c;
      reach = __reduce_add_sync(0xffffffffu, reach);
      uint32_t* w = wthr + (bit & 1) * BM_MWARPS;  // two sets of words in turn: one barrier a bit
      if (lane == 0) w[warp] = reach;
      __syncthreads();
      reach = 0;
#pragma unroll
      for (int i = 0; i < BM_MWARPS; ++i) reach += w[i];
      if (reach >= K) lo = c;
      if (reach >= K && reach <= BM_RANK_CAP) break;
    }
    for (int i = tid; i < n; i += BM_MTHREADS)
      if ((uint32_t)(cs[i] >> 32) >= lo) {
        const int at = atomicAdd(&nsel, 1);
        if (at < BM_RANK_CAP) sel[at] = (unsigned short)i;
      }
    __syncthreads();
    n = nsel;
  }
  const size_t out0 = (size_t)grp * K;
  if (n <= BM_RANK_CAP) {
    for (int i0 = 0; i0 < n; i0 += BM_MTHREADS / 8) {  // eight lanes a candidate
      const int i = i0 + (tid >> 3), me = i < n ? many ? sel[i] : i : 0;
      const uint64_t mine = cs[me];
      const int idx = ci[me];
      int rank = 0;
#pragma unroll 4
      for (int j0 = tid & 7; j0 < n; j0 += 8) {
        const int j = many ? sel[j0] : j0;
        rank += (int)(cs[j] > mine) | ((int)(cs[j] == mine) & (int)(ci[j] < idx));
      }
#pragma unroll
      for (int d = 4; d; d >>= 1) rank += __shfl_xor_sync(0xffffffffu, rank, d);
      if (i < n && (tid & 7) == 0 && rank < K) {
        out_score[out0 + rank] = (float)unord_d(mine);
        out_parent[out0 + rank] = idx / V;
        out_token[out0 + rank] = idx % V;
      }
    }
    for (int i = n + tid; i < K; i += BM_MTHREADS) {
      out_score[out0 + i] = -CUDART_INF_F;
      out_parent[out0 + i] = out_token[out0 + i] = -1;
    }
    return;
  }
  // head by head: K rounds, each taking the best head; a thread keeps the best of its own lists (list l < B * parts, then one
  // entry for each finished beam)
  const int L = B * parts;
  for (int i = tid; i < L + B; i += BM_MTHREADS) taken[i] = 0;
  __syncthreads();
  auto head = [&](int l) -> BeamBest {
    BeamBest r{0.0, 0, -1};
    const int b = l < L ? l / parts : l - L, i = taken[l];
    if (l >= L) {
      if (fin[b] && i == 0 && off[b] == off[b]) r = BeamBest{off[b], b * V + end_token, l};
    } else if (!fin[b] && i < K && off[b] == off[b]) {
      const int2 e = __ldcg(list_of(b, l % parts) + i);
      const float x = __int_as_float(e.x);
      if (x > -CUDART_INF_F) r = BeamBest{score_of(b, x), b * V + e.y, l};
    }
    return r;
  };
  auto mine = [&]() {
    BeamBest r{0.0, 0, -1};
    for (int l = tid; l < L + B; l += BM_MTHREADS) {
      const BeamBest h = head(l);
      if (better(h, r)) r = h;
    }
    return r;
  };
  BeamBest own = mine();
  for (int k = 0; k < K; ++k) {
    BeamBest r = own;
#pragma unroll
    for (int d = 16; d; d >>= 1) {
      const BeamBest o = shfl_best(r, d);
      if (better(o, r)) r = o;
    }
    if (lane == 0) wbest[warp] = r;
    __syncthreads();
    r = wbest[0];
#pragma unroll
    for (int w = 1; w < BM_MWARPS; ++w)
      if (better(wbest[w], r)) r = wbest[w];
    if (tid == 0) {  // (there are more than K candidates)
      out_score[out0 + k] = (float)r.score;
      out_parent[out0 + k] = r.idx / V;
      out_token[out0 + k] = r.idx % V;
    }
    if (r.list >= 0 && r.list % BM_MTHREADS == tid) {
      ++taken[r.list];
      own = mine();
    }
    __syncthreads();
  }
}

// Granules a thread: the largest parts that leave a few dozen (a part has a fixed cost of its own, and the merge one of each:
// 8 best of 128000 logits 9.2, 8.1, 8.1 us with 1, 2, 4 granules a thread; of 4 x 128000 11.8, 9.8, 9.3; of 1000 6.9, 6.9, 7.5).
static int beam_it(int rows, int V) {
  for (int it = 4; it > 1; it /= 2)
    if ((long)rows * ((V + 3) / 4 / (BM_THREADS * it) + 1) >= 24) return it;
  return 1;
}
// Parts of a row, whatever its alignment.
static int beam_parts(int it, int V) { return ((V + 3 + 3) / 4 + BM_THREADS * it - 1) / (BM_THREADS * it); }

size_t beam_workspace(int groups, int beams, int V, int K) {
  const int parts = beam_parts(beam_it(groups * beams, V), V);
  return (size_t)groups * beams * parts * (sizeof(float2) + (size_t)K * sizeof(int2));
}

cudaError_t beam_select(const BeamArgs& a, cudaStream_t s) {
  const int rows = a.groups * a.beams, it = beam_it(rows, a.V), parts = beam_parts(it, a.V);
  float2* stats = reinterpret_cast<float2*>(a.ws);
  int2* lists = reinterpret_cast<int2*>(stats + (size_t)rows * parts);
  auto go = [&](auto kern) {
    return launch(kern, dim3(parts, rows), dim3(BM_THREADS), 0, s, a.logits, a.ld, a.V, a.K, a.scores, a.done, stats,
                  lists);
  };
  cudaError_t e = it == 4 ? go(k_beam_parts<4>) : it == 2 ? go(k_beam_parts<2>) : go(k_beam_parts<1>);
  if (e != cudaSuccess) return e;
  const size_t smem = (size_t)a.beams * (parts + 1);
  return launch(k_beam_merge, dim3(a.groups), dim3(BM_MTHREADS), smem, s, a.beams, a.V, a.K, parts, a.scores, a.done,
                a.end_token, stats, lists, a.out_score, a.out_parent, a.out_token);
}

}  // namespace lfm3
