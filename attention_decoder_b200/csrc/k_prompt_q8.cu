// Attention of a prompt chunk over the 8-bit cache, on tcgen05. The chunk's rows see the whole blocks before it as 8-bit codes
// and everything after in bf16 (lfm3_state in include/lfm3.h).
//
// k_kv8_prompt stores the chunk's rows in the cache and lays the slot's keys and values out as bf16 rows [kv head][position]
// that are exact: the codes themselves (integers up to 127) or the bf16 rows. Scales stay outside, three numbers per block of
// 16 keys: x = log2(e) / sqrt(128) * s_k multiplies scores in the exponent's FMA, y = log2(s_v) is added there, so that P holds
// p * s_v without another operation, and z = 1 / s_v takes it out of the row's sum, once per block. P is rounded to bf16 (2^-8
// relative a probability, averaged over the keys), everything else is fp32.
//
// k_kv8_prompt_attn: a block owns 64 query rows x the 4 query heads of one kv head as two M = 128 tiles, A and B (MMA row
// m = 4 r + head), and a range of 128-key tiles. Warps 0..3 are the softmax of A, 4..7 of B, one thread a row; warp 8 loads K
// and V tiles by TMA (two stages each), warp 9 issues the MMAs: while one tile's scores are in the softmax the other's products
// run. Scores and then P (as the A operand of P V) share TMEM columns 0..127 (A) and 128..255 (B), the outputs hold 256..511.
// MMAs of one thread run in order, so the scores of the next tile overwrite P only when P V has read it. The running maximum
// moves only when a score exceeds it by more than 8 (in log2 units), so that the outputs are hardly ever rescaled.
// An SM does 4096 bf16 MACs and 16 ex2 a clock: 2048 clocks a pair of tiles either way. It takes 3400: a tile's chain of softmax
// (1860, half of it ex2, the rest the warps' other instructions) and products (1100 to 1500) is longer than that, and two tiles
// do not fill it. 2048 rows at 6144 138 us in all (870 TFLOP/s), 777 at 0 23 us, 300 at 1024 24.5 us, 64 at 6000 29 us. Scores
// against the maximum of the tiles before: 140 us otherwise; two issuing warps 193 us; a cubic instead of ex2 for a quarter
// of the pairs 134 us, for half of them 141 us (issue slots); steps of 64 keys, whose half of the columns is refilled while the
// other is in the softmax, 148 us (products of 64 keys): not taken.
#include <cudaTypedefs.h>
#include <algorithm>

#include "kernels.cuh"

namespace lfm3 {

constexpr int PA_ROWS = 64, PA_KT = 128;
constexpr int PA_HALVES = 2;  // parts in which P is handed over (one part: 143.7 us, two: 137.6)
constexpr uint32_t PA_TILE = 128 * HD * 2;  // bytes of a Q, K or V tile of 128 rows: two halves of 64 dims
constexpr int PA_THREADS = 384;  // three warpgroups; the third is the loader, the MMA issuer and two idle warps
constexpr size_t PA_SMEM = 1024 + 6 * PA_TILE + 256;  // Q x 2, two stages of K and V, barriers

DEVI void pa_load(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
DEVI void pa_load_q(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
DEVI void pa_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
DEVI void pa_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// 128-byte-swizzled operand tiles. K-major: rows of 128 B in 8-row atoms of 1024 B.
DEVI uint64_t pa_desc_k(uint32_t a) {
  return (uint64_t)((a >> 4) & 0x3FFFu) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) |
         ((uint64_t)2 << 61);
}
// MN-major: 64 dims per 128-B row, the next 64 dims half a tile later.
DEVI uint64_t pa_desc_mn(uint32_t a) {
  return (uint64_t)((a >> 4) & 0x3FFFu) | ((uint64_t)((PA_TILE / 2) >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
DEVI void pa_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
               "l"(a), "l"(b), "r"(idesc), "r"(accum));
}
DEVI void pa_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
               "r"(a), "l"(b), "r"(idesc), "r"(accum));
}
DEVI bool pa_elect() {  // one lane of a converged warp
  uint32_t e;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.b32 %0, 1, 0, p;\n}" : "=r"(e));
  return e != 0;
}
DEVI void pa_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
DEVI void pa_ld32(uint32_t t, float* v) {  // 32 columns of this warp's lanes; pa_wait_ld() before use
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%"
      "19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(t));
}
DEVI void pa_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
DEVI void pa_st32(uint32_t t, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(t),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
DEVI void pa_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
DEVI float pa_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

DEVI float pa_max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// Pairs of fp32 in one instruction.
DEVI uint64_t pa_pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
DEVI void pa_unpair(uint64_t p, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p)); }
DEVI uint64_t pa_fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
DEVI uint64_t pa_add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__global__ void __launch_bounds__(PA_THREADS, 1)
    k_kv8_prompt_attn(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                      const __grid_constant__ CUtensorMap tv, const Q8PromptAttn a) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t qs = su32(smem), ks = qs + 2 * PA_TILE, vs = ks + 2 * PA_TILE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + 6 * PA_TILE);
  const uint32_t q_full = su32(bars), kv_full = q_full + 8, kv_empty = kv_full + 16, s_full = kv_empty + 16,
                 p_full = s_full + 16, o_done = p_full + 32;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 17);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the last query rows see the most keys: their blocks are dispatched first
  const int kvh = blockIdx.y, pb = gridDim.x - 1 - blockIdx.x, rb0 = pb * PA_ROWS, split = blockIdx.z;
  const int khi = a.p0 + min(a.n, rb0 + PA_ROWS) - 1;         // last key that a row of the block sees
  const int all = khi / PA_KT + 1;                            // tiles up to it
  const int t0 = (int)((long long)all * split / gridDim.z), t1 = (int)((long long)all * (split + 1) / gridDim.z);
  const int nt = t1 - t0;                                     // (none in some splits of the blocks with few)

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(kv_full + 8 * s, 1);
      mbar_init(kv_empty + 8 * s, 1);
      mbar_init(s_full + 8 * s, 1);
      mbar_init(p_full + 16 * s, 4);
      mbar_init(p_full + 16 * s + 8, 4);
      mbar_init(o_done + 8 * s, 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tk)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tv)) : "memory");
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(tmem_slot)), "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  pa_before();
  __syncthreads();
  pa_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_launch_dependents();

  // registers: 384 x 168 at launch; 256 x 216 + 128 x 72 from here on
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
  if (warp == 8) {
    // ---------------------------------------------------------------- loader
    if (lane == 0 && nt > 0) {
      mbar_expect_tx(q_full, 2 * PA_TILE);
      for (int t = 0; t < 2; ++t)
        for (int db = 0; db < 2; ++db)
          pa_load_q(qs + t * PA_TILE + db * (PA_TILE / 2), &tq, db * 64, kvh * GQA, rb0 + 32 * t, q_full);
      int j = 0;
      bool ok = true;
      for (; j < nt; ++j) {
        const int st = j & 1, y = kvh * a.row_pitch + (t0 + j) * PA_KT;
        ok = mbar_wait(kv_empty + 8 * st, ((j >> 1) & 1) ^ 1, a.err);
        if (!ok) break;
        mbar_expect_tx(kv_full + 8 * st, 2 * PA_TILE);
        for (int db = 0; db < 2; ++db) pa_load(ks + st * PA_TILE + db * (PA_TILE / 2), &tk, db * 64, y, kv_full + 8 * st);
        for (int db = 0; db < 2; ++db) pa_load(vs + st * PA_TILE + db * (PA_TILE / 2), &tv, db * 64, y, kv_full + 8 * st);
      }
      if (!ok) {  // the tiles that are on their way land before the block ends (bounded)
        mbar_wait(q_full, 0, a.err);
        for (int i = j < 2 ? 0 : j - 2; i < j; ++i) mbar_wait(kv_full + 8 * (i & 1), (i >> 1) & 1, a.err);
      }
    }
  } else if (warp == 9) {
    // ---------------------------------------------------------------- MMA issuer: the warp waits, one elected lane issues
    constexpr uint32_t idesc_s = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(PA_KT >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
    constexpr uint32_t idesc_o = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((uint32_t)(HD >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
    const uint64_t dq = pa_desc_k(qs), dk = pa_desc_k(ks), dv = pa_desc_mn(vs);  // tiles lie PA_TILE / 16 apart
    auto scores = [&](int t, int st) {  // S of tile t = Q K^T
      if (pa_elect()) {
        const uint64_t qd = dq + t * (PA_TILE / 16), kd = dk + st * (PA_TILE / 16);
#pragma unroll
        for (int k = 0; k < HD / 16; ++k) {
          const uint32_t off = (k >> 2) * (PA_TILE / 32) + (k & 3) * 2;
          pa_mma_ss(tmem + t * 128, qd + off, kd + off, idesc_s, k != 0);
        }
        pa_commit(s_full + 8 * t);
      }
      __syncwarp();
    };
    bool ok = nt > 0 && mbar_wait(q_full, 0, a.err) && mbar_wait(kv_full, 0, a.err);
    if (ok) {
      pa_after();
      scores(0, 0);
      scores(1, 0);
    }
    for (int j = 0; j < nt && ok; ++j) {
      const int st = j & 1, sn = st ^ 1;
      const uint64_t vd = dv + st * (PA_TILE / 16);
      const bool more = j + 1 < nt;
      if (more) ok = mbar_wait(kv_full + 8 * sn, ((j + 1) >> 1) & 1, a.err);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int half = 0; half < PA_HALVES; ++half) {  // P comes in parts of the keys
          ok = ok && mbar_wait(p_full + 16 * t + 8 * half, j & 1, a.err);
          if (!ok) break;
          pa_after();
          if (pa_elect()) {
#pragma unroll
            for (int i = 0; i < PA_KT / 16 / PA_HALVES; ++i) {
              const int k = half * (PA_KT / 16 / PA_HALVES) + i;
              pa_mma_ts(tmem + 256 + t * 128, tmem + t * 128 + k * 8, vd + k * 128, idesc_o, (j | k) != 0);
            }
            // (a stage that no later tile takes is not given back: nothing would wait for that arrival)
            if (half == PA_HALVES - 1 && t == 1 && j + 2 < nt) pa_commit(kv_empty + 8 * st);
            if (half == PA_HALVES - 1 && !more) pa_commit(o_done + 8 * t);
          }
          __syncwarp();
        }
        if (more && ok) scores(t, sn);
      }
    }
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    // ---------------------------------------------------------------- softmax, one thread a row
    const int t = warp >> 2, quarter = warp & 3, m = quarter * 32 + lane;
    const int r = rb0 + 32 * t + (m >> 2), h = kvh * GQA + (m & 3), qp = a.p0 + r;
    const int dense_hi = a.p0 + rb0 + 32 * t;  // keys up to here are seen by every row of the tile
    const uint32_t ts = tmem + ((uint32_t)(quarter * 32) << 16) + t * 128, to = ts + 256;
    float mrun = -INFINITY, lrun = 0.f;
    bool ok = true;
    for (int j = 0; j < nt && ok; ++j) {
      const int kt0 = (t0 + j) * PA_KT;
      const float4* blk = a.blk + (size_t)kvh * (a.row_pitch / QBLK) + kt0 / QBLK;
      float4 c[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] = __ldcg(blk + i);
      ok = __all_sync(0xffffffffu, mbar_wait(s_full + 8 * t, j & 1, a.err));
      if (!ok) break;
      pa_after();
      float v[128];
#pragma unroll
      for (int i = 0; i < 4; ++i) pa_ld32(ts + 32 * i, v + 32 * i);
      pa_wait_ld();
      const bool dense = kt0 + PA_KT - 1 <= dense_hi;
      if (!dense) {
#pragma unroll
        for (int i = 0; i < 128; ++i)
          if (kt0 + i > qp) v[i] = -INFINITY;
      }
      uint32_t pk[32];
      float l = lrun, mu = mrun == -INFINITY ? 0.f : mrun;
      // probabilities of keys 16 b0 .. 16 b1 - 1 into pk, and their sum
      auto probabilities = [&](auto B0, auto B1, auto masked) {
        constexpr int b0 = decltype(B0)::value, b1 = decltype(B1)::value;
#pragma unroll
        for (int b = b0; b < b1; ++b) {
          const float add = c[b].y - mu;
          const uint64_t mul2 = pa_pair(c[b].x, c[b].x), add2 = pa_pair(add, add);
          uint64_t sum = 0, sum1 = 0;
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            float p0, p1;
            pa_unpair(pa_fma2(pa_pair(v[16 * b + i], v[16 * b + i + 1]), mul2, add2), p0, p1);
            p0 = pa_ex2(p0);
            p1 = pa_ex2(p1);
            if constexpr (decltype(masked)::value) {  // (a scale of 0 or NaN would turn a masked score into NaN)
              if (kt0 + 16 * b + i > qp) p0 = 0.f;
              if (kt0 + 16 * b + i + 1 > qp) p1 = 0.f;
            }
            if (i & 2)
              sum1 = pa_add2(sum1, pa_pair(p0, p1));
            else
              sum = pa_add2(sum, pa_pair(p0, p1));
            pk[8 * (b - b0) + i / 2] = pack_bf2(p0, p1);
          }
          float s0, s1;
          pa_unpair(pa_add2(sum, sum1), s0, s1);
          l = fmaf(s0 + s1, c[b].z, l);
        }
      };
      using F = std::integral_constant<int, 0>;
      using H = std::integral_constant<int, 4>;
      using E = std::integral_constant<int, 8>;
      // the first half of the probabilities against the maximum of the tiles before, while the tile's own is found
      if (dense)
        probabilities(F{}, H{}, std::false_type{});
      float tmax = -INFINITY;
#pragma unroll
      for (int b = 0; b < 8; ++b) {
        const float* w = v + 16 * b;
        const float m0 = pa_max3(w[0], w[1], w[2]), m1 = pa_max3(w[3], w[4], w[5]), m2 = pa_max3(w[6], w[7], w[8]),
                    m3 = pa_max3(w[9], w[10], w[11]), m4 = pa_max3(w[12], w[13], w[14]);
        tmax = fmaxf(tmax, pa_max3(pa_max3(m0, m1, m2), pa_max3(m3, m4, w[15]), -INFINITY) * c[b].x);
      }
      const bool grows = tmax > mrun + 8.f;
      if (__any_sync(0xffffffffu, grows) || !dense) {
        const float mnew = grows ? tmax : mrun;
        mu = mnew == -INFINITY ? 0.f : mnew;
        const float alpha = pa_ex2(mrun - mu);
        if (__any_sync(0xffffffffu, j > 0 && alpha < 1.f)) {  // P V of the tiles before has finished: it precedes these scores
#pragma unroll 1
          for (int i = 0; i < 4; ++i) {
            float o[32];
            pa_ld32(to + 32 * i, o);
            pa_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] *= alpha;
            pa_st32(to + 32 * i, reinterpret_cast<uint32_t*>(o));
          }
        }
        mrun = mnew;
        l = lrun * alpha;
        probabilities(F{}, H{}, std::true_type{});
      }
      auto hand_over = [&](int half) {
        pa_st32(ts + 32 * half, pk);
        pa_wait_st();
        if (half == 1 || PA_HALVES == 2) {
          pa_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full + 16 * t + (PA_HALVES == 2 ? 8 * half : 0));
        }
      };
      hand_over(0);
      if (dense)
        probabilities(H{}, E{}, std::false_type{});
      else
        probabilities(H{}, E{}, std::true_type{});
      hand_over(1);
      lrun = l;
    }
    ok = ok && nt > 0 && __all_sync(0xffffffffu, mbar_wait(o_done + 8 * t, 0, a.err));
    if (ok) {
      pa_after();
      const bool live = r < a.n;
      const size_t prow = (((size_t)pb * HKV + kvh) * gridDim.z + split) * 256 + t * 128 + m;
      const float gt = live && gridDim.z == 1 ? sigmoidf_(__ldcg(a.gate + (size_t)r * HQ + h)) / lrun : 1.f;
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {
        float o[32];
        pa_ld32(to + 32 * i, o);
        pa_wait_ld();
        if (gridDim.z == 1) {
          if (live) {
            uint4* d = reinterpret_cast<uint4*>(a.y + ((size_t)r * HQ + h) * HD + 32 * i);
#pragma unroll
            for (int q = 0; q < 4; ++q)
              d[q] = make_uint4(pack_bf2(o[8 * q] * gt, o[8 * q + 1] * gt), pack_bf2(o[8 * q + 2] * gt, o[8 * q + 3] * gt),
                                pack_bf2(o[8 * q + 4] * gt, o[8 * q + 5] * gt), pack_bf2(o[8 * q + 6] * gt, o[8 * q + 7] * gt));
          }
        } else {
          float4* d = reinterpret_cast<float4*>(a.part + prow * HD + 32 * i);
#pragma unroll
          for (int q = 0; q < 8; ++q) d[q] = make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
        }
      }
      if (gridDim.z > 1) a.part_ml[prow] = make_float2(mrun, lrun);
    } else if (gridDim.z > 1) {
      const size_t prow = (((size_t)pb * HKV + kvh) * gridDim.z + split) * 256 + t * 128 + m;
      a.part_ml[prow] = make_float2(-INFINITY, 0.f);
    }
  }
  pa_before();
  __syncthreads();
  pa_after();
  if (warp == 9) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
}

// The splits of a row: warp = (row, query head); blocks of the four heads of one kv head. Latency bounds it: one or a few rounds
// of eight loads in flight. (Merging in the block that came last instead: 9 rows at 6080 56 us in all, not 25.)
__global__ void __launch_bounds__(128) k_kv8_prompt_merge(const Q8PromptAttn a, int ns) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, head = threadIdx.x >> 5, r = blockIdx.x, kvh = blockIdx.y;
  const size_t base = ((size_t)(r / PA_ROWS) * HKV + kvh) * ns * 256 + r % PA_ROWS / 32 * 128 + r % 32 * 4 + head;
  const float gate = __ldcg(a.gate + (size_t)r * HQ + kvh * GQA + head);
  float M = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0; s0 < ns; s0 += 8) {
    float2 ml[8];
    float4 x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const size_t at = base + (size_t)min(s0 + e, ns - 1) * 256;
      ml[e] = __ldcg(a.part_ml + at);
      x[e] = __ldcg(reinterpret_cast<const float4*>(a.part + at * HD) + lane);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      // a split that saw no key of this row has a sum of 0 (and nothing written); one that saw only NaN scores has a
      // maximum of -inf and a sum of NaN, which counts
      if (s0 + e >= ns || ml[e].y == 0.f) continue;
      const float m = ml[e].x == -INFINITY ? M : fmaxf(M, ml[e].x);
      const float keep = M == -INFINITY ? (l != l ? 1.f : 0.f) : pa_ex2(M - m), w = ml[e].x == -INFINITY ? 1.f : pa_ex2(ml[e].x - m);
      M = m;
      l = l * keep + w * ml[e].y;
      acc.x = acc.x * keep + w * x[e].x;
      acc.y = acc.y * keep + w * x[e].y;
      acc.z = acc.z * keep + w * x[e].z;
      acc.w = acc.w * keep + w * x[e].w;
    }
  }
  const float gt = sigmoidf_(gate) / l;
  reinterpret_cast<uint2*>(a.y + ((size_t)r * HQ + kvh * GQA + head) * HD)[lane] =
      make_uint2(pack_bf2(acc.x * gt, acc.y * gt), pack_bf2(acc.z * gt, acc.w * gt));
}

// Splits over the keys: none while the rows give every SM a block; then as many as fit on the SMs, of at least two tiles of the
// middle row (a split costs a block's start, a partial result and its share of the merge). 64 rows at 6000 104 us with one,
// 29 with 23; at least two, three or four tiles of the last row instead: 777 rows at 0 (now one split) 28.8, 28.8, 23.1 us, 300 at
// 1024 24.6, 26.0, 29.4 (now 24.5), 600 at 500 27.5, 27.5, 30.7 (27.4), 64 at 512 22.1, 21.1, 21.1 (21.9). More than fit at once,
// in two rounds: 1300 rows at 6000 122 -> 111 us, but 1500 at 2000 66 -> 75.
static int kv8_prompt_splits(int p0, int n) {
  const int blocks = (n + PA_ROWS - 1) / PA_ROWS * HKV;
  return std::max(1, std::min(PA_BLOCKS / blocks, (p0 + n / 2) / (2 * PA_KT)));
}

cudaError_t kv8_prompt_attn(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const Q8PromptAttn& a,
                            cudaStream_t s) {
  const int ns = kv8_prompt_splits(a.p0, a.n);
  const cudaError_t e = launch(k_kv8_prompt_attn, dim3((a.n + PA_ROWS - 1) / PA_ROWS, HKV, ns), dim3(PA_THREADS), PA_SMEM, s, tq,
                               tk, tv, a);
  return e != cudaSuccess || ns == 1 ? e : launch(k_kv8_prompt_merge, dim3(a.n, HKV), dim3(128), 0, s, a, ns);
}

cudaError_t kv8_prompt_init() {
  return cudaFuncSetAttribute(k_kv8_prompt_attn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)PA_SMEM);
}

// bf16 rows [rows][128] in boxes of 128 rows x 64 dims, 128-byte swizzle.
bool make_tmap_rows128(CUtensorMap* m, const void* base, uint64_t rows) {
  static PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
  if (!enc) {
    cudaDriverEntryPointQueryResult q;
    void* fn = nullptr;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || fn == nullptr)
      return false;
    enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }
  cuuint64_t dims[2] = {HD, rows};
  cuuint64_t strides[1] = {HD * 2};
  cuuint32_t box[2] = {64, 128};
  cuuint32_t es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace lfm3
