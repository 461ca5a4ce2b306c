// The order in which a warp of k_kv8_attend looks tiles up and loads them, apart from where its lanes run (the host compiles
// this too). No CUDA headers.
#pragma once

#ifdef __CUDACC__
#define Q8_HD __device__ __forceinline__
#else
#define Q8_HD inline
#endif

namespace lfm3 {

// Tiles 0 .. n - 1 of a share, looked up 32 at a time and up to a batch ahead of the tile that is attended. B: what look-ups of
// 32 tiles gave, B::row(i) the row of the i-th in the pool (-1: nothing to load, which every look-up behind the share gives).
template <class B>
struct Q8Ahead {
  B cur, nxt;  // the batch of the present tile, and the one behind it once its first tile is done
  // Row of tile k, which lies in the batch of the present tile or in the next one.
  Q8_HD int row(int k, int present) const { return ((k ^ present) & ~31 ? nxt : cur).row(k & 31); }
  // Tile k is done. (The next batch is looked up even if the share has nothing there: what is left of an older one would be
  // loaded, into memory that nobody waits for.)
  template <class L>
  Q8_HD void done(int k, const L& look_up) {
    if ((k & 31) == 0) nxt = look_up(k + 32);
    if ((k & 31) == 31) cur = nxt;
  }
};

}  // namespace lfm3
