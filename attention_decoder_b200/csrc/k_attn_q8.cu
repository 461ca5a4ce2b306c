// Attention of a full layer over the 8-bit cache (layout and rounding: lfm3_state in include/lfm3.h).
//
// A key or value is s * c with c an int8 code and s one scale per 16 positions and kv head, so a tile of 16 positions
// is exactly one m16 operand of the warp MMA and its scale leaves the product: q.k = s_k (q.c), and the tile's share of
// the output is s_v (p.c). The codes become f16 operands without rounding (1024 + 128 + c is put together by byte
// permutes, 1152 subtracted in f16), the sums stay fp32. Queries are bf16 values held in f16 (exact from 2^-14 to
// 65504 in size). Probabilities, relative to the warp's reference, are rounded to f16 after a factor of 2^7: 2^-11 relative
// (against the output's bf16 2^-8) for those of 2^-21 and more, below that 2^-32 absolute a key, 2^-14 in all for the 2^18
// keys that a warp has at most. The block that a row lies in itself is attended in bf16 from the tail ring, its probabilities
// split into two bf16 halves (2^-16).
//
// Decode (k_kv8_attend): HBM bounds it at 1026 bytes a key and layer (4 heads x 256 B of codes + 2 B of scales). One
// grid of resident blocks takes shares of all pages x kv heads of the batch, whatever the streams' lengths: whole shares of
// one (stream, kv head) segment a block, or equal shares in order. Where a segment has several blocks, the parts merge through
// global memory by a tree of eights, each step in the block that comes last. All rows of a stream's window (groups of four)
// share a segment, so a code is read once for them: the MMA's 8 columns are (row, query head) pairs. Each of a block's four
// warps owns one quarter of every page, i.e. whole 16-key tiles, streams them by TMA through its own ring of buffers across
// segment borders (evict-first in L2: read once, and the lengths, tables, queries and parts stay), and keeps its own online
// softmax; they meet only where a segment ends, while the SM's other blocks keep the memory busy.
// Measured (one layer, graph of calls over three caches): one stream at 2047 keys 10.7 us, at 131000 34.6 us (134 MB, 3.9 TB/s),
// 64 streams at 256..8191 59.3 us (278 MB, 4.7 TB/s), at 8000 96 us (526 MB, 5.5 TB/s), 13 windows of 4 rows at 500..8100 27.4 us.
// 64 streams at 8000 take 39.5 us more than at 4000: 6.7 TB/s while it streams. The rest is latency: 4 us to the first tile
// (lengths, table, tile: three dependent reads), 6 to 8 us of merges behind the last, 2 to 4 us at a second segment. Windows
// are bound by the warps' instructions (two n-tiles: 8 warps an SM).
#include <cudaTypedefs.h>
#include <climits>

#include "kernels.cuh"
#include "q8_ahead.cuh"

namespace lfm3 {

constexpr int Q8_WARPS = 4, Q8_THREADS = 32 * Q8_WARPS;
constexpr int Q8_TILE = QBLK * HD;  // bytes of a tile of codes, K or V
// A block's share, in pages, where there is little to share: fewer parts have fewer levels of merges, more parts shorter loops. With
// 2, 3, 4 pages one stream takes at 300 keys 8.3, 8.9, 8.9 us, at 1000 8.7, 9.0, 9.9, at 2047 10.9, 10.8, 10.8, at 4000 10.4, 11.2, 11.2;
// 4 streams at 2047 12.8, 12.3, 11.8; 2 windows of 3 rows at 3300..5200 16.0, 17.0, 16.7.
constexpr int Q8_MIN_PAGES = 2;
static_assert(PAGE == Q8_WARPS * QBLK, "a warp owns one quarter of every page");

DEVI void q8_tma(uint32_t dst, const CUtensorMap* map, int row, uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(bar), "l"(policy)
      : "memory");
}
DEVI uint4 lds16(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
  return r;
}
DEVI uint32_t movmatrix_t(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
DEVI float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Bytes (code + 128) at places 0, 1 (lo) or 2, 3 (hi) of w -> f16x2 of the codes.
DEVI uint32_t codes_lo(uint32_t w) {
  const uint32_t m = __byte_perm(w, 0x64646464u, 0x4140);
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(0x64806480u));
  return r;
}
DEVI uint32_t codes_hi(uint32_t w) {
  const uint32_t m = __byte_perm(w, 0x64646464u, 0x4342);
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(0x64806480u));
  return r;
}
DEVI uint32_t pack_h2(float lo, float hi) {
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}
DEVI uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Codes of values x with scale s, without a division each. x and s are bf16 values, so x / s is either a multiple of 1/2 or
// at least 2^-11 away from the nearest odd multiple (its denominator is below 2^8, or 2^10 where it lies under 1), while
// x * (1 / s) in fp32 is off by less than 2^-16: put on the grid of 2^-12 first, it is rounded to the integer that the
// exact quotient is rounded to, ties to even included.
struct Q8Scale {
  float s, lift, inv;
  uint32_t keep;
  // The scale of a block whose largest magnitude is a: a / 127 rounded up to a bf16 value. (Denormal scales and their values
  // are lifted by 2^64 first, which is exact.)
  DEVI Q8Scale(float a, bool bad) {
    s = __uint_as_float((__float_as_uint(__fdiv_rn(a, 127.f)) + 0xFFFFu) & 0xFFFF0000u);
    lift = s < 1e-30f ? 18446744073709551616.f : 1.f;
    inv = s > 0.f ? __frcp_rn(s * lift) : 0.f;
    keep = bad ? 0u : ~0u;  // a block that is not finite has codes of 0
  }
  DEVI uint32_t code(float x) const {
    const float grid = __fadd_rn(__fadd_rn(x * lift * inv, 2560.f), -2560.f);  // ulp(2560) = 2^-12
    return __float_as_uint(__fadd_rn(grid, 12582912.f)) & 0xFFu;               // ulp(1.5 * 2^23) = 1
  }
  DEVI uint32_t codes(uint2 w) const {
    return (code(bflo(w.x)) | code(bfhi(w.x)) << 8 | code(bflo(w.y)) << 16 | code(bfhi(w.y)) << 24) & keep;
  }
};

// Where row `pos` of a stream is: this pass's own rows from p0 on, or the tail ring.
struct TailRow {
  const bf16 *ring, *fresh;  // ring of (slot, kv head); row 0 of this pass (HKV * HD elements a row)
  int p0;
  DEVI const bf16* at(int pos) const {
    return pos >= p0 ? fresh + (size_t)(pos - p0) * HKV * HD : ring + (size_t)(pos % QRING) * HD;
  }
};

// The scale of a full block of 16 rows that a warp holds (lane l: dims 4l .. + 3 of each).
DEVI Q8Scale q8_scale(const uint2 (&x)[QBLK], float* stored) {
  float a = 0.f;
  bool bad = false;
#pragma unroll
  for (int r = 0; r < QBLK; ++r) {
    const float v[4] = {bflo(x[r].x), bfhi(x[r].x), bflo(x[r].y), bfhi(x[r].y)};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      a = fmaxf(a, fabsf(v[k]));
      bad |= !(fabsf(v[k]) < INFINITY);
    }
  }
  a = warp_max(a);
  bad = __any_sync(0xffffffffu, bad);
  const Q8Scale s(a, bad);
  *stored = bad ? __uint_as_float(0x7fc00000u) : s.s;
  return s;
}
DEVI Q8Scale q8_rows(const TailRow& t, int first, uint2 (&x)[QBLK], int lane, float* stored) {  // reads them first
#pragma unroll
  for (int r = 0; r < QBLK; ++r) x[r] = __ldcg(reinterpret_cast<const uint2*>(t.at(first + r)) + lane);
  return q8_scale(x, stored);
}

// A pass's rows of one stream and kv head, keys or values, into the ring, and the block that they fill into 8 bits: a warp. (The
// pass's other readers do not see what is written here: neither that block's codes, nor ring rows of positions from p0 on,
// which are less than 32 away from those that they read.)
DEVI void q8_store_rows(const Q8Attend& A, int stream, int kvh, int isv, int lane) {
  const int slot = __ldcg(A.d_slots + stream), p0 = __ldcg(A.seq_len + slot), b0 = p0 / QBLK;
  bf16* tail = (isv ? A.tail_v : A.tail_k) + ((size_t)slot * HKV + kvh) * QRING * HD;
  const TailRow R{tail, (isv ? A.v : A.k) + ((size_t)stream * A.W * HKV + kvh) * HD, p0};
  if ((p0 + A.W) / QBLK > b0) {
    const int page = __ldcg(A.table + (size_t)slot * A.max_pages + p0 / PAGE);
    const size_t tile = (size_t)page * HKV + kvh;
    uint2 x[QBLK];
    float stored;
    const Q8Scale s = q8_rows(R, b0 * QBLK, x, lane, &stored);
    int8_t* dst = (isv ? A.vq : A.kq) + (tile * PAGE + (b0 & 3) * QBLK) * HD;
#pragma unroll
    for (int i = 0; i < QBLK; ++i) reinterpret_cast<uint32_t*>(dst + i * HD)[lane] = s.codes(x[i]);
    if (lane == 0) (isv ? A.v_scale : A.k_scale)[tile * (PAGE / QBLK) + (b0 & 3)] = stored;
  }
  for (int i = 0; i < A.W; ++i)
    reinterpret_cast<uint2*>(tail + (size_t)((p0 + i) % QRING) * HD)[lane] = __ldcg(reinterpret_cast<const uint2*>(R.at(p0 + i)) + lane);
}

// NT: n-tiles of 8 columns = 2 rows x 4 heads each. Two of them take 254 registers, so two blocks an SM (three, with 300 bytes
// spilled, made 13 windows of 4 rows half as long again). A fourth tile in flight does not help (3 % slower).
// SEGMENT: 3, 4, 6, 8 pages gave 63.1, 62.5, 62.8, 64.1 us for 64 streams at 256..8191 and 33.5, 31.8, 30.8, 30.8 for 3 at
// 23000..43000; with two n-tiles 6, 10, 12 pages gave 30.5, 28.8, 28.8 for 13 windows of 4 rows.
template <int NT>
struct Q8Shape {
  static constexpr int RESIDENT = NT == 1 ? 3 : 2;  // blocks per SM
  static constexpr int DEPTH = 3;                        // tiles in flight per warp
  static constexpr int COLS = 8 * NT;
  static constexpr int SEGMENT = NT == 1 ? 6 : 10;  // what a second segment costs a block, in pages
  static constexpr int RING = Q8_WARPS * DEPTH * 2 * Q8_TILE;
  static constexpr int QTILE = COLS * HD * 2;
  static constexpr int SMEM = 1024 + RING + 2 * Q8_TILE + QTILE + Q8_WARPS * COLS * HD * 4;  // + the tile that a window fills, + states
};

template <int NT>
__global__ void __launch_bounds__(Q8_THREADS, Q8Shape<NT>::RESIDENT)
    k_kv8_attend(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const Q8Attend A) {
  using S = Q8Shape<NT>;
  constexpr int D = S::DEPTH;
  extern __shared__ __align__(1024) unsigned char dsm[];
  __shared__ __align__(8) uint64_t bars[Q8_WARPS][D];
  __shared__ float wm[Q8_WARPS][S::COLS], wl[Q8_WARPS][S::COLS];
  __shared__ int pre[65], slots[64], lens[64];  // page-heads before stream i; its slot; its position p0
  __shared__ int last, smin[Q8_WARPS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const uint32_t smem0 = (su32(dsm) + 1023u) & ~1023u;
  const uint32_t base = smem0 + warp * (D * 2 * Q8_TILE), made_tile = smem0 + S::RING, qtile = made_tile + 2 * Q8_TILE;
  float* obuf = reinterpret_cast<float*>(dsm + (smem0 - su32(dsm)) + S::RING + 2 * Q8_TILE + S::QTILE);  // [warp][column][HD]
  uint64_t policy;  // codes are read once: what else the step reads stays in L2
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  if (lane == 0) {
    for (int k = 0; k < D; ++k) mbar_init(su32(&bars[warp][k]), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    if (warp == 0) {
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tk)) : "memory");
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tv)) : "memory");
    }
  }
  __syncwarp();
  pdl_wait();
  pdl_launch_dependents();
  // two blocks a stream behind the others store its rows: a warp for each head's keys and values
  const int G = gridDim.x - 2 * A.streams;
  if ((int)blockIdx.x >= G) {
    const int u = (blockIdx.x - G) * Q8_WARPS + warp;
    q8_store_rows(A, u / (2 * HKV), u / 2 % HKV, u & 1, lane);
    return;
  }

  // ---- the work list: streams in order, each with HKV x groups segments (kv head, row group) of its pages, from the last
  // page (with the open block) to the first: a sequence of page-heads.
  if (warp < 2) {
    const int i = tid;
    int n = 0;
    if (i < A.streams) {
      slots[i] = __ldcg(A.d_slots + i);
      lens[i] = __ldcg(A.seq_len + slots[i]);
      n = ((lens[i] + A.W - 1) / PAGE + 1) * HKV * A.groups;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, n, o);
      if (lane >= o) n += v;
    }
    pre[i + 1] = n;
    if (i == 0) pre[0] = 0;
  }
  __syncthreads();
  auto pages_of = [&](int s) -> int { return (lens[s] + A.W - 1) / PAGE + 1; };
  const int hg = HKV * A.groups, blk = blockIdx.x;
  const int P = A.streams > 32 ? pre[32] + pre[A.streams] : pre[A.streams];
  // A block for whole shares of one segment: of `per` pages at most, the fewest with which the blocks suffice ..
  const int n0 = lane < A.streams ? pages_of(lane) : 0, n1 = lane + 32 < A.streams ? pages_of(lane + 32) : 0;  // (this lane's)
  {
    // .. if that is no more than a block's part (in pages, a further segment's cost included) of equal shares. 61 streams at
    // 51..86 take 11.4 us with whole shares, 20 with equal ones. 64 at 256..8191 take 80 us with whole shares (of 54 pages), 68
    // with equal ones (of 42). (There are more blocks than segments, so `per` = P would do for any batch.)
    const int least = max(Q8_MIN_PAGES, (P + G - 1) / G), most = P < 2 * G ? P : (P + S::SEGMENT * hg * A.streams) / G;
    int found = INT_MAX;
    for (int s = least + warp; s <= most && found == INT_MAX; s += Q8_WARPS)
      if (hg * __reduce_add_sync(0xffffffffu, (n0 + s - 1) / s + (n1 + s - 1) / s) <= G) found = s;
    if (lane == 0) smin[warp] = found;
  }
  if (A.streams > 32) {
    __syncthreads();
    if (warp == 1 && lane < A.streams - 32) pre[33 + lane] += pre[32];
  }
  __syncthreads();
  int per = INT_MAX;
#pragma unroll
  for (int w = 0; w < Q8_WARPS; ++w) per = min(per, smin[w]);
  const bool whole = per != INT_MAX;
  const int PW = P + S::SEGMENT * hg * A.streams;
  struct Place { int stream, hg, page, pages; };
  int lo, hi, my_parts = 0, my_part = 0;  // this block's page-heads; with whole shares, its segment's blocks and its place
  Place mine{0, 0, 0, 0};                 // with whole shares: its segment (page: that of page-head 0)
  if (whole) {
    const int b0 = hg * ((n0 + per - 1) / per), b1 = hg * ((n1 + per - 1) / per);
    int e0 = b0, e1 = b1;  // blocks up to and with stream `lane`, `lane + 32`
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, e0, o), b = __shfl_up_sync(0xffffffffu, e1, o);
      if (lane >= o) e0 += a, e1 += b;
    }
    e1 += __shfl_sync(0xffffffffu, e0, 31);
    const int s = __popc(__ballot_sync(0xffffffffu, e0 <= blk)) + __popc(__ballot_sync(0xffffffffu, e1 <= blk));
    if (s >= A.streams) return;
    const int i = blk - __shfl_sync(0xffffffffu, s < 32 ? e0 - b0 : e1 - b1, s & 31), n = pages_of(s);
    my_parts = (n + per - 1) / per;
    mine = Place{s, i / my_parts, 0, n};
    my_part = i - mine.hg * my_parts;
    lo = pre[s] + mine.hg * n;
    mine.page = n - 1 + lo;
    hi = lo + (int)((unsigned)n * (my_part + 1) / my_parts);  // (at most 444 parts: no overflow below 2^22 pages)
    lo += (int)((unsigned)n * my_part / my_parts);
  } else {
    // Equal shares count a segment's fixed cost as SEGMENT pages: weight w(x) = x + SEGMENT (segments up to x's) of page-head x.
    auto first_at = [&](int w) -> int {  // page-heads of less weight than w
      int s = 0;
#pragma unroll
      for (int d = 32; d; d >>= 1)
        if (s + d < A.streams && pre[s + d] + S::SEGMENT * hg * (s + d) <= w) s += d;
      const int n = pages_of(s), i = w - pre[s] - S::SEGMENT * hg * s;
      return pre[s] + i / (n + S::SEGMENT) * n + max(0, i % (n + S::SEGMENT) - S::SEGMENT);
    };
    lo = first_at((int)((long long)blk * PW / G));
    hi = blk + 1 == G ? P : first_at((int)((long long)(blk + 1) * PW / G));
  }
  auto block_of = [&](int x, int segments) -> int {  // (equal shares) the block with page-head x, of so many segments up to it
    return (int)(((long long)(x + S::SEGMENT * segments + 1) * G - 1) / PW);
  };

  auto find = [&](int r) -> Place {  // page-head r
    Place f = mine;
    if (whole) {
      f.page -= r;
      return f;
    }
    int s = 0;
#pragma unroll
    for (int d = 32; d; d >>= 1)
      if (s + d < A.streams && pre[s + d] <= r) s += d;
    f.stream = s;
    f.pages = pages_of(s);
    const int i = r - pre[s];
    f.hg = i / f.pages;
    f.page = f.pages - 1 - i % f.pages;
    return f;
  };
  // Tile k of this warp: quarter `warp` of page-head lo + k. Lanes look 32 tiles up at a time, up to a batch ahead (Q8Ahead):
  // the row of the tile in the pool (-1: not a tile of codes, or behind the share) and its scales.
  struct Batch {
    int at;
    float ks, vs;
    DEVI int row(int i) const { return __shfl_sync(0xffffffffu, at, i); }
  };
  auto look_up = [&](int k0) -> Batch {
    Batch x{-1, 0.f, 0.f};
    const int r = lo + k0 + lane;
    if (r < hi) {
      const Place f = find(r);
      if (4 * f.page + warp < lens[f.stream] / QBLK) {
        const int page = __ldcg(A.table + (size_t)slots[f.stream] * A.max_pages + f.page);
        const int tile = page * HKV + f.hg / A.groups;
        x.at = tile * PAGE + warp * QBLK;
        x.ks = __ldcg(A.k_scale + (size_t)tile * (PAGE / QBLK) + warp);
        x.vs = __ldcg(A.v_scale + (size_t)tile * (PAGE / QBLK) + warp);
      }
    }
    return x;
  };
  // Queries, held in f16: column n = g of n-tile j is (row r0 + 2j + n / 4, head 4 kvh + n % 4). The MMA's k index i of lane t
  // stands for dims 32 t + 4 i .. + 3 (any order of the dims will do as long as keys and queries agree on it), so chunk x of
  // a column lies at place x % 4 of lane (g, x / 4). A segment's are requested ahead of the tiles that its block waits
  // for: behind them they would take as long.
  const uint32_t qplace = (((tid & 3) * 32 + (tid >> 4) * 4 + ((tid & 15) >> 2)) * 16);  // of chunk tid % 16 of column tid / 16
  auto request_q = [&](const Place& f) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int col = tid >> 4, rr = f.hg % A.groups * 2 * NT + 2 * j + (col >> 2), row = f.stream * A.W + min(rr, A.W - 1);
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(qtile + j * (Q8_THREADS * 16) + qplace),
                   "l"(A.q + ((size_t)row * HQ + f.hg / A.groups * GQA + (col & 3)) * HD + 8 * (tid & 15)), "r"(rr < A.W ? 16 : 0)
                   : "memory");
    }
  };
  if (lo < hi) request_q(find(lo));
  Q8Ahead<Batch> ahead{look_up(0), Batch{-1, 0.f, 0.f}};
  auto fetch = [&](int k, int present, int place) {  // tile k into that ring place
    const int row = ahead.row(k, present);
    if (row >= 0 && lane == 0) {
      const uint32_t bar = su32(&bars[warp][place]), dst = base + place * 2 * Q8_TILE;
      mbar_expect_tx(bar, 2 * Q8_TILE);
      q8_tma(dst, &tk, row, bar, policy);
      q8_tma(dst + Q8_TILE, &tv, row, bar, policy);
    }
  };
  for (int k = 0; k < D; ++k) fetch(k, 0, k);
  uint32_t par = 0;  // phase of each ring slot's barrier
  const float sl2 = rsqrtf((float)HD) * 1.4426950408889634f;  // scores in base 2
  constexpr float P_DOWN = 0x1p-7f;  // takes P_UP = 2^7 out again: with the values' scale, in the tail and in the sums
  bool ok = true;
  int k = 0, at = 0;  // tile, its place in the ring
  for (int r = lo; r < hi;) {  // segments
    const Place f = find(r);
    const int seg0 = pre[f.stream] + f.hg * f.pages, seg1 = seg0 + f.pages, end = min(seg1, hi);
    const int slot = slots[f.stream], p0 = lens[f.stream], kvh = f.hg / A.groups, r0 = f.hg % A.groups * 2 * NT;
    const int nr = min(A.W - r0, 2 * NT), pr = p0 + r0;  // rows of this segment, position of the first
    const int blast = (pr + nr - 1) / QBLK, bfirst = pr / QBLK;  // own blocks of the last and first row
    const int b0 = p0 / QBLK;                                     // the block that was open before the pass
    const size_t row0 = (size_t)f.stream * A.W;

    // queries: each thread converts its chunks; one n-tile's then stay in registers
    asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const uint32_t at = qtile + j * (Q8_THREADS * 16) + qplace;
      const uint4 w = lds16(at);
      asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(bf2_to_h2(w.x)), "r"(bf2_to_h2(w.y)), "r"(bf2_to_h2(w.z)),
                   "r"(bf2_to_h2(w.w))
                   : "memory");
    }
    __syncthreads();
    uint4 qf[4];
    if constexpr (NT == 1) {
#pragma unroll
      for (int c = 0; c < 4; ++c) qf[c] = lds16(qtile + (c * 32 + lane) * 16);
    }
    int own[NT];  // own block of the row that this lane's columns 2t, 2t + 1 belong to
#pragma unroll
    for (int j = 0; j < NT; ++j) own[j] = (pr + min(2 * j + (t >> 1), nr - 1)) / QBLK;

    float o[NT][8][4];               // rows: dims 16 g + 2 i, + 1; columns 2t, 2t + 1
    float mrun[NT][2], lrun[NT][2];  // per column: reference, 7 below a score (P_UP), and this lane's keys' sum
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int i = 0; i < 8; ++i) o[j][i][0] = o[j][i][1] = o[j][i][2] = o[j][i][3] = 0.f;
      mrun[j][0] = mrun[j][1] = -INFINITY;
      lrun[j][0] = lrun[j][1] = 0.f;
    }
    // Online softmax of one tile's scores c (base 2, masked to -inf): c becomes the probabilities times P_UP. The reference that
    // is subtracted moves, and o is rescaled, only when a score is more than 8 above the one it was made of (times P_UP, that is
    // 2^15, within f16), so that most tiles need one vote instead of a maximum over the lanes.
    auto softmax = [&](float (&c)[NT][4]) {
      bool grows = false;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) grows |= fmaxf(c[j][e], c[j][2 + e]) - mrun[j][e] > 15.f;
      if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float m = fmaxf(c[j][e], c[j][2 + e]);
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
            m = fmaxf(m - 7.f, mrun[j][e]);
            const float al = m == -INFINITY ? 1.f : ex2(mrun[j][e] - m);
            mrun[j][e] = m;
            lrun[j][e] *= al;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              o[j][i][e] *= al;
              o[j][i][2 + e] *= al;
            }
          }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float ref = mrun[j][e] == -INFINITY ? 0.f : mrun[j][e];  // nothing visible yet: all probabilities are 0
          c[j][e] = ex2(c[j][e] - ref);
          c[j][2 + e] = ex2(c[j][2 + e] - ref);
          lrun[j][e] += c[j][e] + c[j][2 + e];
        }
    };
    const size_t ring = ((size_t)slot * HKV + kvh) * QRING * HD, fresh = (row0 * HKV + kvh) * HD;
    const TailRow K{A.tail_k + ring, A.k + fresh, p0}, V{A.tail_v + ring, A.v + fresh, p0};

    // a tile of codes, block u; every: all rows of the segment see it
    auto tile = [&](uint32_t kt, float ks, float vs, int u, auto every) {
      const uint32_t vt = kt + Q8_TILE;
      ks *= sl2;
      vs *= P_DOWN;
      float c[NT][4], c2[NT][4];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) c[j][e] = c2[j][e] = 0.f;
      // keys g and g + 8 (the 128-byte swizzle moves 16-byte chunk x of row r to x ^ (r & 7))
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t off = (uint32_t)g * HD + (((2 * t + h) ^ (g & 7)) << 4);
        const uint4 ka = lds16(kt + off), kb = lds16(kt + off + 8 * HD);
        uint4 qh[NT][2];  // the k steps' queries
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int c = 0; c < 2; ++c)
            if constexpr (NT == 1)
              qh[j][c] = qf[2 * h + c];
            else
              qh[j][c] = lds16(qtile + ((j * 4 + 2 * h + c) * 32 + lane) * 16);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t xa = word(ka, w) ^ 0x80808080u, xb = word(kb, w) ^ 0x80808080u;
          const uint32_t a0 = codes_lo(xa), a1 = codes_lo(xb), a2 = codes_hi(xa), a3 = codes_hi(xb);
#pragma unroll
          for (int j = 0; j < NT; ++j)
            mma_f16_16816(w & 1 ? c2[j] : c[j], a0, a1, a2, a3, word(qh[j][w >> 1], 2 * (w & 1)), word(qh[j][w >> 1], 2 * (w & 1) + 1));
        }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) c[j][e] = decltype(every)::value || u < own[j] ? (c[j][e] + c2[j][e]) * ks : -INFINITY;
      softmax(c);
      uint32_t pf[NT][2];
      float vsj[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        pf[j][0] = movmatrix_t(pack_h2(c[j][0], c[j][1]));
        pf[j][1] = movmatrix_t(pack_h2(c[j][2], c[j][3]));
        vsj[j] = decltype(every)::value || u < own[j] ? vs : 0.f;  // a block that the row does not see in 8 bits adds nothing, whatever its scale
      }
      // dims 16 g .. + 15 of keys 2t, 2t + 1, 2t + 8, 2t + 9
      const uint32_t r1 = 2 * t, voff = r1 * HD + ((g ^ r1) << 4), voff1 = (r1 + 1) * HD + ((g ^ (r1 + 1)) << 4);
      const uint4 va = lds16(vt + voff), vb = lds16(vt + voff1), vc = lds16(vt + voff + 8 * HD), vd = lds16(vt + voff1 + 8 * HD);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t xa = word(va, w) ^ 0x80808080u, xb = word(vb, w) ^ 0x80808080u;
        const uint32_t xc = word(vc, w) ^ 0x80808080u, xd = word(vd, w) ^ 0x80808080u;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t y1 = __byte_perm(xa, xb, h ? 0x7362 : 0x5140), y2 = __byte_perm(xc, xd, h ? 0x7362 : 0x5140);
          const uint32_t a0 = codes_lo(y1), a1 = codes_hi(y1), a2 = codes_lo(y2), a3 = codes_hi(y2);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            float d[4] = {0.f, 0.f, 0.f, 0.f};
            mma_f16_16816(d, a0, a1, a2, a3, pf[j][0], pf[j][1]);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][2 * w + h][e] += vsj[j] * d[e];
          }
        }
      }
      __syncwarp();  // the buffer is read
    };

    // ---- this warp's tiles of the segment
    auto next_tile = [&]() {
      ahead.done(k, look_up);
      ++k;
      at = at + 1 == D ? 0 : at + 1;
    };
    for (; lo + k < end; next_tile()) {  // those with the rows' own blocks and behind
      const int u = 4 * (seg1 - 1 - (lo + k)) + warp;  // the tile's block of 16 positions
      if (u < b0) break;
      if (u == b0 && b0 < blast) {
        // a window that runs into the next block shows its later rows this one in 8 bits: its tile is built here
        float ks, vs;
        uint2 x[QBLK];
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv) {
          const Q8Scale s = q8_rows(kv ? V : K, b0 * QBLK, x, lane, kv ? &vs : &ks);
#pragma unroll
          for (int i = 0; i < QBLK; ++i)
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(made_tile + kv * Q8_TILE + i * HD + (((lane >> 2) ^ (i & 7)) << 4) + 4 * (lane & 3)),
                         "r"(s.codes(x[i]))
                         : "memory");
        }
        __syncwarp();
        if (ok) tile(made_tile, ks, vs, u, std::false_type{});
      }
      if (ok) fetch(k + D, k, at);
      if (u >= bfirst && u <= blast) {  // an open block, in bf16
        const int first = u * QBLK, n = min(QBLK, pr + nr - first);  // written rows that the segment may see
        // (rows past the last are read as the last one: loads that depend on nothing are in flight together)
        const uint4 z = make_uint4(0, 0, 0, 0);
        const uint4* k0 = reinterpret_cast<const uint4*>(K.at(first + min(g, n - 1)) + 32 * t);
        const uint4* k1 = reinterpret_cast<const uint4*>(K.at(first + min(g + 8, n - 1)) + 32 * t);
        uint4 x0[4], x1[4];
#pragma unroll
        for (int cc = 0; cc < 4; ++cc) {
          x0[cc] = __ldcg(k0 + cc);
          x1[cc] = __ldcg(k1 + cc);
        }
        float c[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          c[j][0] = c[j][1] = c[j][2] = c[j][3] = 0.f;
          const int rr = 2 * j + (g >> 2);
          const uint4* qp = reinterpret_cast<const uint4*>(A.q + ((row0 + r0 + min(rr, nr - 1)) * HQ + kvh * GQA + (g & 3)) * HD + 32 * t);
          uint4 q[4];  // (a column without a row: another's, and not used)
#pragma unroll
          for (int cc = 0; cc < 4; ++cc) q[cc] = __ldcg(qp + cc);
#pragma unroll
          for (int cc = 0; cc < 4; ++cc) {
            mma_bf16_16816(c[j], x0[cc].x, x1[cc].x, x0[cc].y, x1[cc].y, q[cc].x, q[cc].y);
            mma_bf16_16816(c[j], x0[cc].z, x1[cc].z, x0[cc].w, x1[cc].w, q[cc].z, q[cc].w);
          }
        }
        // values of keys 2t, 2t + 1, 2t + 8, 2t + 9, dims 16 g .. + 15. One that is not finite counts as zeros with a score of
        // NaN, so that it reaches the rows that see its key and no others.
        uint4 vr[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4* vp = reinterpret_cast<const uint4*>(V.at(first + min(2 * t + (i & 1) + 8 * (i >> 1), n - 1)) + 16 * g);
          vr[i][0] = __ldcg(vp);
          vr[i][1] = __ldcg(vp + 1);
        }
        uint32_t bad = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t e = 0;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int w = 0; w < 4; ++w) e |= ((word(vr[i][h], w) & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
          bad |= (e ? 1u : 0u) << i;
        }
        bad |= __shfl_xor_sync(0xffffffffu, bad, 4);
        bad |= __shfl_xor_sync(0xffffffffu, bad, 8);
        bad |= __shfl_xor_sync(0xffffffffu, bad, 16);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if ((bad >> i & 1) || 2 * t + (i & 1) + 8 * (i >> 1) >= n) vr[i][0] = vr[i][1] = z;
        const uint32_t badk = __shfl_sync(0xffffffffu, bad, g >> 1) >> (g & 1);  // bit 0: key g, bit 2: key g + 8
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const int seen = own[j] == u ? pr + min(2 * j + (t >> 1), nr - 1) - first : -1;  // last key that the row sees
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (badk >> (e & 2) & 1) c[j][e] = __uint_as_float(0x7fc00000u);
            c[j][e] = g + 8 * (e >> 1) <= seen ? c[j][e] * sl2 : -INFINITY;
          }
        }
        softmax(c);
        uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float p = c[j][2 * e] * P_DOWN, q = c[j][2 * e + 1] * P_DOWN, hp = round_bf(p), hq = round_bf(q);
            ph[j][e] = movmatrix_t(pack_bf2(hp, hq));
            pl[j][e] = movmatrix_t(pack_bf2(p - hp, q - hq));
          }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 va = vr[0][h], vb = vr[1][h], vc = vr[2][h], vd = vr[3][h];
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t a0 = __byte_perm(word(va, w), word(vb, w), 0x5410), a1 = __byte_perm(word(va, w), word(vb, w), 0x7632);
            const uint32_t a2 = __byte_perm(word(vc, w), word(vd, w), 0x5410), a3 = __byte_perm(word(vc, w), word(vd, w), 0x7632);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              mma_bf16_16816(o[j][4 * h + w], a0, a1, a2, a3, ph[j][0], ph[j][1]);
              mma_bf16_16816(o[j][4 * h + w], a0, a1, a2, a3, pl[j][0], pl[j][1]);
            }
          }
        }
      }
    }
    // the rest, in a loop of its own (no masks, no other code between). 64 streams at 256..8191 take 59.2 us instead of 63.1, windows
    // 7 % less; one stream at 2047 keys takes 10.6 instead of 9.9 (4 of the 1017 us of a whole token).
    for (; lo + k < end; next_tile()) {
      if (!ok) continue;
      ok = __all_sync(0xffffffffu, mbar_wait(su32(&bars[warp][at]), (par >> at) & 1, A.err));
      if (!ok) continue;
      par ^= 1u << at;
      tile(base + at * 2 * Q8_TILE, __shfl_sync(0xffffffffu, ahead.cur.ks, k & 31), __shfl_sync(0xffffffffu, ahead.cur.vs, k & 31), 0, std::true_type{});
      fetch(k + D, k, at);
    }

    // ---- the warps' states merge: columns' sums over the lanes, then exp2(M_w - M) weights
    if (r != lo) __syncthreads();  // the last segment's states are read
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l = lrun[j][e];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        const int col = 8 * j + 2 * t + e;
        if (g == 0) {
          // NaN scores leave the maximum alone: a warp that saw nothing else still has to count
          wm[warp][col] = l != l ? fmaxf(mrun[j][e], 0.f) : mrun[j][e];
          wl[warp][col] = l * P_DOWN;  // (as the outputs: relative to the reference and P_UP, the same for all states)
        }
        if (col < 4 * nr) {
          float* ob = obuf + ((size_t)warp * S::COLS + col) * HD + 16 * g;
#pragma unroll
          for (int i = 0; i < 8; ++i) *reinterpret_cast<float2*>(ob + 2 * i) = make_float2(o[j][i][e], o[j][i][2 + e]);
        }
      }
    __syncthreads();
    if (end < hi) request_q(find(end));
    const int nseg = f.stream * hg + f.hg + 1;
    int nact = my_parts, part = my_part;  // blocks of this segment, and this one's place among them
    if (!whole) {
      const int first_blk = block_of(seg0, nseg);
      nact = block_of(seg1 - 1, nseg) - first_blk + 1;
      part = blk - first_blk;
    }
    const int ncol = 4 * nr;
    const size_t mloff = (size_t)A.rows * HQ * A.nsp * HD;
    auto row_head = [&](int col) -> size_t {  // (row, query head) of a column
      return (row0 + r0 + (col >> 2)) * HQ + kvh * GQA + (col & 3);
    };
    auto put = [&](size_t rh, const float4& o, float l) {  // a finished row and head
      const float gt = sigmoidf_(__ldcg(A.gate + rh)) / l;
      reinterpret_cast<uint2*>(A.y + rh * HD)[lane] = make_uint2(pack_bf2(o.x * gt, o.y * gt), pack_bf2(o.z * gt, o.w * gt));
    };
    for (int col = warp; col < ncol; col += Q8_WARPS) {  // a warp takes a column
      float M = -INFINITY, l = 0.f;
#pragma unroll
      for (int w = 0; w < Q8_WARPS; ++w) M = fmaxf(M, wm[w][col]);
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < Q8_WARPS; ++w) {
        const float wt = wm[w][col] == -INFINITY ? 0.f : ex2(wm[w][col] - M);
        const float4 x = *reinterpret_cast<const float4*>(obuf + ((size_t)w * S::COLS + col) * HD + 4 * lane);
        s.x += wt * x.x; s.y += wt * x.y; s.z += wt * x.z; s.w += wt * x.w;
        l += wt * wl[w][col];
      }
      const size_t rh = row_head(col);
      if (nact == 1) {
        put(rh, s, l);
      } else {
        reinterpret_cast<float4*>(A.part + (rh * A.nsp + part) * HD)[lane] = s;
        if (lane == 0) *reinterpret_cast<float2*>(A.part + mloff + 2 * (rh * A.nsp + part)) = make_float2(M, l);
      }
    }
    if (nact > 1) {
      // parts merge by a tree: the last block of eight neighbours merges theirs (in place, in the first one's slot), the last
      // such block of the segment merges the eights
      float2* ml = reinterpret_cast<float2*>(A.part + mloff);
      unsigned* count = A.counters + (((size_t)f.stream * A.groups + f.hg % A.groups) * HKV + kvh) * Q8_COUNTERS;
      auto is_last = [&](unsigned* c, int of) -> bool {
        __syncthreads();
        if (tid == 0) {
          unsigned old;
          asm volatile("atom.add.acq_rel.gpu.u32 %0, [%1], 1;" : "=r"(old) : "l"(c) : "memory");
          last = old == (unsigned)(of - 1);
          if (last) *c = 0u;
        }
        __syncthreads();
        return last;
      };
      auto merge = [&](int first, int step, int n, bool final) {  // parts first + i * step, i < n; a warp takes NT columns
        for (int col0 = NT * warp; col0 < ncol; col0 += NT * Q8_WARPS) {
          size_t hb[NT];
          float M[NT], l[NT];
          float4 acc[NT];
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            hb[j] = row_head(min(col0 + j, ncol - 1)) * A.nsp + first;
            M[j] = -INFINITY;
            l[j] = 0.f;
            acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
          }
          for (int s0 = 0; s0 < n; s0 += 8) {
            float2 m2[NT][8];
            float4 x[NT][8];
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const size_t at = hb[j] + (size_t)min(s0 + e, n - 1) * step;  // (past the last: the last one, with no weight)
                m2[j][e] = __ldcg(&ml[at]);
                x[j][e] = __ldcg(reinterpret_cast<const float4*>(A.part + at * HD) + lane);
              }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if (s0 + e >= n) {
                  m2[j][e] = make_float2(-INFINITY, 0.f);
                  x[j][e] = make_float4(0.f, 0.f, 0.f, 0.f);
                }
              float Mn = M[j];
#pragma unroll
              for (int e = 0; e < 8; ++e) Mn = fmaxf(Mn, m2[j][e].x);
              const float al = M[j] == -INFINITY ? 0.f : ex2(M[j] - Mn);
              float4& a = acc[j];
              l[j] *= al;
              a.x *= al; a.y *= al; a.z *= al; a.w *= al;
              M[j] = Mn;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float wt = m2[j][e].x == -INFINITY ? 0.f : ex2(m2[j][e].x - Mn);
                l[j] += wt * m2[j][e].y;
                a.x += wt * x[j][e].x; a.y += wt * x[j][e].y; a.z += wt * x[j][e].z; a.w += wt * x[j][e].w;
              }
            }
          }
          __syncwarp();  // every lane has read the parts' maxima and sums
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            if (col0 + j >= ncol) break;
            if (final) {
              put(row_head(col0 + j), acc[j], l[j]);
            } else {
              reinterpret_cast<float4*>(A.part + hb[j] * HD)[lane] = acc[j];
              if (lane == 0) ml[hb[j]] = make_float2(M[j], l[j]);
            }
          }
        }
      };
      const int eights = (nact + 7) / 8, mine = part / 8, n = min(8, nact - 8 * mine);
      if (is_last(count + 1 + mine, n)) {
        merge(8 * mine, 1, n, eights == 1);
        if (eights > 1 && is_last(count, eights)) merge(0, 8, eights, true);
      }
    }
    r = end;
  }
  if (!ok && lane == 0)  // copies still in flight land before the block exits (bounded)
    for (int i = 0; i < D; ++i) mbar_wait(su32(&bars[warp][i]), (par >> i) & 1, A.err);
}

// ------------------------------------------------------------------------------------------ prompt chunks
// Rows at positions p0 .. p0 + n - 1 of one slot (k, v: bf16 [n][HKV][HD]) enter the cache, and the slot's keys and values are
// laid out for k_kv8_prompt_attn, exactly (but see factors): codes before the chunk's first block, the open block's and the
// chunk's own rows, and zeros up to the end of the last tile of 128. A value row that is not finite is laid out as zeros with a key of NaN, so that
// the rows that see it become NaN and masked ones do not.
// Warp (block of 16 positions, kv head, K or V; K's and V's are neighbours). A block that becomes full is stored as codes; rows
// of a last block that does not go to the ring. The first block reads ring rows that the last one may overwrite (blocks an
// even number apart share them), so one pair of warps does both, in that order (the warp of K reads values too). HBM bounds it (512 B of codes
// a position in, 1 KB out); 8192 positions took 3.7 us (the loads of a block all in flight: 12 us one at a time).
__global__ void __launch_bounds__(128) k_kv8_prompt(const Q8Prompt A) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5, kvh = blockIdx.y, isv = warp & 1;
  const int p0 = __ldcg(A.seq_len + A.slot), end = p0 + A.n;
  const int t0 = p0 / QBLK, t1 = (end - 1) / QBLK;
  int t = blockIdx.x * 2 + (warp >> 1);
  if (t * QBLK >= A.row_pitch || (t == t1 && t1 != t0)) return;  // the last block: see below
  const int32_t* table = A.table + (size_t)A.slot * A.max_pages;
  const size_t ring = ((size_t)A.slot * HKV + kvh) * QRING * HD;
  int8_t* codes = isv ? A.vq : A.kq;
  float* scales = isv ? A.v_scale : A.k_scale;
  bf16* rows = (isv ? A.rows_v : A.rows_k) + (size_t)kvh * A.row_pitch * HD;
  float* blk = reinterpret_cast<float*>(A.blk + (size_t)kvh * (A.row_pitch / QBLK));
  const TailRow K{A.tail_k + ring, A.k + kvh * HD, p0}, V{A.tail_v + ring, A.v + kvh * HD, p0};
  const TailRow& R = isv ? V : K;
  bf16* tail = (isv ? A.tail_v : A.tail_k) + ring;
  const float sl2 = rsqrtf((float)HD) * 1.4426950408889634f;
  // The factors of a block, from its scale. A scale of values outside 2^-60 .. 2^100 would leave probabilities times it no room
  // in a float: the excess, which is returned, goes into the values (rounded to bf16 then).
  auto factors = [&](int block, float s) -> float {
    float rest = 1.f;
    if (isv) {
      if (s == 0.f) s = 1.f;  // a block of zeros
      const float in = s < 0x1p-60f ? 0x1p-60f : s > 0x1p100f ? 0x1p100f : s;
      if (in != s && s == s) rest = s < in ? s * 0x1p60f : s * 0x1p-100f;
      if (lane == 0) {
        *reinterpret_cast<float2*>(blk + 4 * block + 2) = make_float2(1.f / in, 0.f);
        blk[4 * block + 1] = log2f(in);
      }
    } else if (lane == 0) {
      blk[4 * block] = sl2 * s;
    }
    return rest;
  };
  for (;; t = t1) {
    const int first = t * QBLK, sub = first % PAGE;
    bf16* out = rows + (size_t)first * HD;
    const int n = max(0, min(QBLK, end - first));  // rows there are
    if (t < t0) {
      const size_t tile = (size_t)__ldcg(table + first / PAGE) * HKV + kvh;
      const float scale = __ldcg(scales + tile * (PAGE / QBLK) + sub / QBLK);
      const uint32_t* src = reinterpret_cast<const uint32_t*>(codes + (tile * PAGE + sub) * HD) + lane;
      uint32_t w[QBLK];
#pragma unroll
      for (int r = 0; r < QBLK; ++r) w[r] = __ldcg(src + r * (HD / 4));
      const float rest = factors(t, scale);
#pragma unroll
      for (int r = 0; r < QBLK; ++r) {
        float x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = (float)(int8_t)(w[r] >> (8 * k)) * rest;
        reinterpret_cast<uint2*>(out + r * HD)[lane] = make_uint2(pack_bf2(x[0], x[1]), pack_bf2(x[2], x[3]));
      }
      return;
    }
    factors(t, 1.f);
    const uint2 z = make_uint2(0, 0);
    uint2 x[QBLK], v[QBLK];  // the rows, and their values (rows past the end: the last one's, so that no load has to wait)
    const int top = end - 1;
#pragma unroll
    for (int r = 0; r < QBLK; ++r) x[r] = __ldcg(reinterpret_cast<const uint2*>(R.at(min(first + r, top))) + lane);
#pragma unroll
    for (int r = 0; r < QBLK; ++r) v[r] = __ldcg(reinterpret_cast<const uint2*>(V.at(min(first + r, top))) + lane);
    uint32_t bad = 0;  // rows whose values are not finite
#pragma unroll
    for (int r = 0; r < QBLK; ++r) {
      if (r >= n) x[r] = z;
      const uint2 y = r < n ? v[r] : z;
      // all ones in a bf16 exponent: the sum with its lowest bit carries into the sign
      const uint32_t e = (((y.x & 0x7f807f80u) + 0x00800080u) | ((y.y & 0x7f807f80u) + 0x00800080u)) & 0x80008000u;
      bad |= (e ? 1u : 0u) << r;
    }
    bad = __reduce_or_sync(0xffffffffu, bad);
#pragma unroll
    for (int r = 0; r < QBLK; ++r)
      reinterpret_cast<uint2*>(out + r * HD)[lane] = !(bad >> r & 1) ? x[r] : isv ? z : make_uint2(0x7fc07fc0u, 0x7fc07fc0u);
    if (n == QBLK) {
      const size_t tile = (size_t)__ldcg(table + first / PAGE) * HKV + kvh;
      float stored;
      const Q8Scale s = q8_scale(x, &stored);
#pragma unroll
      for (int r = 0; r < QBLK; ++r) reinterpret_cast<uint32_t*>(codes + (tile * PAGE + sub + r) * HD)[lane] = s.codes(x[r]);
      if (lane == 0) scales[tile * (PAGE / QBLK) + sub / QBLK] = stored;
    } else {  // the open block at the chunk's end
#pragma unroll
      for (int r = 0; r < QBLK; ++r)
        if (r < n && first + r >= p0) reinterpret_cast<uint2*>(tail + (size_t)((first + r) % QRING) * HD)[lane] = x[r];
    }
    if (t != t0 || t1 == t0) return;
    asm volatile("bar.sync %0, 64;" ::"r"(1 + (warp >> 1)) : "memory");  // both warps have read the ring
  }
}

cudaError_t kv8_prompt_rows(const Q8Prompt& a, int p0, cudaStream_t s) {
  const int blocks = (p0 + a.n + 127) / 128 * (128 / QBLK);
  return launch(k_kv8_prompt, dim3((blocks + 1) / 2, HKV), dim3(128), 0, s, a);
}

int kv8_blocks(int W) { return 148 * (W <= 2 ? Q8Shape<1>::RESIDENT : Q8Shape<2>::RESIDENT); }

cudaError_t kv8_attend(const CUtensorMap& tk, const CUtensorMap& tv, Q8Attend a, cudaStream_t s) {
  static_assert(148 * Q8Shape<1>::RESIDENT <= 8 * (Q8_COUNTERS - 1), "a counter for every eight parts of a segment");
  a.groups = (a.W + 3) / 4;  // of up to four rows
  static_assert(2 * HKV == 2 * Q8_WARPS, "a stream's keys and values in two blocks");
  const dim3 grid(kv8_blocks(a.W) + 2 * a.streams), block(Q8_THREADS);
  // one n-tile for 1 and 2 rows: 13 streams at 4000 with 2 rows 20.3 us (two n-tiles: 23.7), with 3 rows 29.5 (25.7)
  return a.W <= 2 ? launch(k_kv8_attend<1>, grid, block, Q8Shape<1>::SMEM, s, tk, tv, a)
                  : launch(k_kv8_attend<2>, grid, block, Q8Shape<2>::SMEM, s, tk, tv, a);
}

cudaError_t kv8_init() {
  const cudaError_t e = cudaFuncSetAttribute(k_kv8_attend<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, Q8Shape<1>::SMEM);
  return e != cudaSuccess ? e
                          : cudaFuncSetAttribute(k_kv8_attend<2>, cudaFuncAttributeMaxDynamicSharedMemorySize, Q8Shape<2>::SMEM);
}

// Codes of one layer's pool viewed as [rows][128 bytes], tiles of 16 rows, 128-byte swizzle.
bool make_tmap_q8(CUtensorMap* m, const void* base, uint64_t rows) {
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
  cuuint64_t strides[1] = {HD};
  cuuint32_t box[2] = {HD, QBLK};
  cuuint32_t es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace lfm3
