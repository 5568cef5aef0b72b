// Low-rank adapters of many requests: out_t = base_t + s_a B_a (A_a x_t) for
// the adapter a of token t, one batch holding tokens of many adapters.
//
// Tokens are gathered by adapter into tiles of up to 16 MT tokens of one
// adapter, so that an adapter's weights are read once per tile:
//   k_plan     (batches above kAdapterScanT = 64) counting sort of the tokens by
//              adapter, and the tile list; smaller batches are gathered by every
//              workgroup for itself: 16.6 us against 17.3 and a launch for 64
//              tokens of 64 adapters, 9.7 against 11.9 for one; from 128 the
//              scan costs more (21.4 against 18.9)
//   k_shrink   z = A_a x for a tile over one range of Kd; the partial sums go
//              to z [range][T][R] in fp32
//   k_expand   z's ranges added in order, scaled, and multiplied by B_a; base
//              is read and out written once
// Both products run on the matrix cores with exact products and fp32
// accumulation: x and the weights as they are, z (fp32) as three bf16 parts
// (24 bits; an fp16 B_a as two), so that nothing between the two products is
// rounded below fp32. A token's arithmetic does not depend on the tile it is
// in: its results are the same in any batch of the same launch shape.
// Rows past an adapter's rank are never read, columns past it never used.
//
// 128 tokens of 64 adapters, 4096 x 4096, ranks up to 32: plan 3.8, shrink 5.9,
// expand 7.3 us, bound by chains of latencies (the tile's tokens, its operands,
// the sums). 4093 tokens of 16 adapters, 2816 x 2816, ranks up to 64: plan 6.2,
// shrink 16.6, expand 32.4 us (19.4 and 33.7 where base and out pass through the
// caches as other data does); the last moves 92 MB of base and out and reads B
// through the cache, 16 bytes a cycle (a fragment's lanes lie in 16 rows).
#include "k_block_common.h"
#include "mpb.h"
#include "mpb_internal.h"

namespace mpb {

namespace {

__device__ __forceinline__ acc4 mfma16(bx8 a, bx8 b, acc4 c) { return mfma(a, b, c); }
__device__ __forceinline__ acc4 mfma16(hx8 a, hx8 b, acc4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// Group of a token: its adapter, or n for none.
__device__ __forceinline__ int group_of(const AdapterParams& p, int t) {
  const int a = p.adapter[t];
  return a >= 0 && a < p.n ? a : p.n;
}

__device__ __forceinline__ int rank_of(const AdapterParams& p, int a) {
  if (a >= p.n) return 0;
  const int r = p.ranks ? p.ranks[a] : p.R;
  return r < 0 ? 0 : r < p.R ? r : p.R;
}

// The tile of a workgroup: its adapter (n: none), the adapter's rank and its
// tokens (toks[i] = -1 past its end).
struct __align__(16) TileLds {
  int ids[kAdapterScanT];
  int toks[64];
  int adapter, rank;
};
static_assert(kAdapterScanT == 64, "one wave scans the batch");

// Finds it; false if there is no such tile.
template <int ROWS>
__device__ __forceinline__ bool find_tile(const AdapterParams& p, int tile, TileLds& s, int& adapter, int& rank) {
  const int tid = threadIdx.x;
  if (p.perm) {  // within the lists' room for any tile
    const int count = p.tiles[0];
    const int* d = p.tiles + 4 + 2 * (size_t)tile;  // adapter, rank
    const int a = d[0], r = d[1], t = tid < ROWS ? p.perm[(size_t)tile * ROWS + tid] : -1;
    if (tile >= count) return false;
    if (tid < ROWS) s.toks[tid] = t;
    adapter = a;
    rank = r;
    __syncthreads();
    return true;
  }
  // the first wave, a lane per token: pos = earlier tokens of the same group;
  // every ROWS-th token of a group starts a tile, tiles numbered by their first token
  if (tid < 64) {
    const int id = tid < p.T ? group_of(p, tid) : -1;
    const int r = id >= 0 ? rank_of(p, id) : 0;  // on its way during the scan
    s.ids[tid] = id;
    s.toks[tid] = -1;
    if (tid == 0) s.adapter = -1;
    __builtin_amdgcn_wave_barrier();  // one wave's LDS accesses run in order
    int pos = 0;
    typedef int ix4 __attribute__((ext_vector_type(4)));
#pragma unroll 4
    for (int i = 0; i < p.T; i += 4) {
      const ix4 v = *(const ix4*)&s.ids[i];
#pragma unroll
      for (int k = 0; k < 4; ++k) pos += i + k < tid && v[k] == id ? 1 : 0;
    }
    const bool first = id >= 0 && pos % ROWS == 0;
    const unsigned long long m = __ballot(first);
    const bool lead = first && __popcll(m & ((1ull << tid) - 1)) == tile;
    const unsigned long long at = __ballot(lead);
    if (at) {
      const int l = __ffsll(at) - 1, a = __shfl(id, l), part = __shfl(pos, l) / ROWS;
      if (id == a && pos / ROWS == part) s.toks[pos % ROWS] = tid;
      if (lead) {
        s.adapter = id;
        s.rank = r;
      }
    }
  }
  __syncthreads();
  adapter = s.adapter;
  rank = s.rank;
  return adapter >= 0;
}

// Counting sort of the tokens by group and the tile list, one workgroup: two
// passes over the ids, eight of a thread's loads at once. A wave whose lanes all
// hold one group (a run of one request's tokens) takes its places together; the
// lanes of others meet at the LDS counters. The order of tokens within a tile is
// whatever the counters give and changes no result.
constexpr int kPlanIds = 8;

__global__ __launch_bounds__(1024) void k_plan(AdapterParams p, int rows) {
  __shared__ int cnt[kAdapterMaxN + 1];
  __shared__ int wsum[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, G = p.n + 1;
  for (int i = tid; i < G; i += 1024) cnt[i] = 0;
  __syncthreads();
  const auto load = [&](int t0, int (&id)[kPlanIds]) {
#pragma unroll
    for (int i = 0; i < kPlanIds; ++i) {
      const int t = t0 + 1024 * i + tid;
      id[i] = group_of(p, t < p.T ? t : p.T - 1);
    }
#pragma unroll
    for (int i = 0; i < kPlanIds; ++i)
      if (t0 + 1024 * i + tid >= p.T) id[i] = -1;
  };
  const auto take = [&](int id) {  // this lane's place among the tokens of its group
    const int g = __builtin_amdgcn_readfirstlane(id);
    if (__ballot(id == g) == ~0ull) {
      int base = 0;
      if (g >= 0 && lane == 0) base = atomicAdd(&cnt[g], 64);
      return __builtin_amdgcn_readfirstlane(base) + lane;
    }
    return id >= 0 ? atomicAdd(&cnt[id], 1) : 0;
  };
  int id[kPlanIds];
  for (int t0 = 0; t0 < p.T; t0 += 1024 * kPlanIds) {
    load(t0, id);
#pragma unroll
    for (int i = 0; i < kPlanIds; ++i)
      if (t0 + 1024 * i < p.T) take(id[i]);
  }
  __syncthreads();
  // first tile of each group: a thread scans a run of groups
  const int per = (G + 1023) / 1024, g0 = tid * per, g1 = g0 + per < G ? g0 + per : G;
  int n = 0;
  for (int g = g0; g < g1; ++g) n += (cnt[g] + rows - 1) / rows;
  int ni = n;  // inclusive over the wave
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int b = __shfl_up(ni, d);
    if (lane >= d) ni += b;
  }
  if (lane == 63) wsum[wave] = ni;
  __syncthreads();
  for (int w = 0; w < wave; ++w) ni += wsum[w];
  int tile = ni - n;
  for (int g = g0; g < g1; ++g) {
    const int k = cnt[g], r = k ? rank_of(p, g) : 0;
    cnt[g] = tile * rows;  // the group's first place
    for (int i = 0; i < k; i += rows, ++tile) {
      p.tiles[4 + 2 * tile] = g;
      p.tiles[5 + 2 * tile] = r;
    }
    for (int i = cnt[g] + k; i < tile * rows; ++i) p.perm[i] = -1;  // places past the last tile's end
  }
  if (tid == 1023) p.tiles[0] = ni;
  __syncthreads();
  for (int t0 = 0; t0 < p.T; t0 += 1024 * kPlanIds) {
    if (p.T > 1024 * kPlanIds) load(t0, id);  // else they are still there
#pragma unroll
    for (int i = 0; i < kPlanIds; ++i) {
      if (t0 + 1024 * i < p.T) {
        const int at = take(id[i]);
        if (id[i] >= 0) p.perm[at] = t0 + 1024 * i + tid;
      }
    }
  }
}

// z of one tile over one range of Kd. The waves take steps of 32 (wide tiles:
// pairs of them, whole cache lines of x) in turn; their sums meet in LDS in a
// fixed order. Wide tiles split Kd over 8 waves rather than over more ranges, whose
// partial sums k_expand would have to read again for every 256 columns. RT: rank
// tiles of 16.
constexpr int shrink_waves(int MT) { return MT == 1 ? 4 : 8; }

template <class D, int MT, int RT>
__global__ __launch_bounds__(64 * shrink_waves(MT)) void k_shrink(AdapterParams p) {
  constexpr int NW = shrink_waves(MT), U = MT == 1 ? 1 : 2;
  typedef typename D::vec vec;
  typedef typename D::elem elem;
  __shared__ TileLds tl;
  __shared__ float sum[4][16 * MT][16 * RT + 1];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = lane & 15, g = lane >> 4;
  int a, rank;
  if (!find_tile<16 * MT>(p, blockIdx.x, tl, a, rank) || rank == 0) return;
  const int steps = p.Kd / (32 * U), s0 = (int)((long long)steps * blockIdx.y / gridDim.y),
            s1 = (int)((long long)steps * (blockIdx.y + 1) / gridDim.y);
  // Loads are unconditional, so that those of several steps go out together:
  // rows past the tile's end repeat its first token and rows past the rank the
  // adapter's first row, and what they give is not used.
  const elem* x[MT];
  const elem* w[RT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int t = tl.toks[16 * m + n];
    x[m] = (const elem*)p.X + (size_t)(t < 0 ? tl.toks[0] : t) * p.Kd + 8 * g;
  }
#pragma unroll
  for (int r = 0; r < RT; ++r)
    w[r] = (const elem*)p.A + ((size_t)a * p.R + (16 * r + n < rank ? 16 * r + n : 0)) * p.Kd + 8 * g;
  acc4 acc[MT][RT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[m][r] = (acc4)(0.0f);
#pragma unroll(MT == 1 ? 4 : 1)
  for (int s = s0 + wave; s < s1; s += NW) {
    vec xv[U][MT], av[U][RT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int m = 0; m < MT; ++m) xv[u][m] = *(const vec*)(x[m] + 32 * (U * s + u));
#pragma unroll
      for (int r = 0; r < RT; ++r) av[u][r] = *(const vec*)(w[r] + 32 * (U * s + u));
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int r = 0; r < RT; ++r) acc[m][r] = mfma16(xv[u][m], av[u][r], acc[m][r]);
  }
  for (int v = 0; v < NW; v += 4) {  // wave w adds to sum w % 4
    if (wave / 4 == v / 4) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float* at = &sum[wave & 3][16 * m + 4 * g + i][16 * r + n];
            *at = v ? *at + acc[m][r][i] : acc[m][r][i];
          }
    }
    __syncthreads();
  }
  float* z = p.z + (size_t)blockIdx.y * p.T * p.R;
  for (int i = tid; i < 16 * MT * 16 * RT; i += 64 * NW) {
    const int row = i / (16 * RT), r = i % (16 * RT), t = tl.toks[row];
    if (t >= 0 && r < p.R) z[(size_t)t * p.R + r] = (sum[0][row][r] + sum[1][row][r]) + (sum[2][row][r] + sum[3][row][r]);
  }
}

// out of one tile: a wave holds 16 tokens and 64 columns at a time. With MT = 4
// the waves take the tile's four rows of 16 tokens, with MT = 1 the columns in
// turn. RK: rank tiles of 32. The columns are the products' rows, so that a
// lane has four consecutive columns of one token; the wave's sums then pass
// through LDS, so that base and out are read and written 256 bytes of a row at a
// time. The next 64 columns' base and B are always on their way, in the other of
// two register sets: the loop holds no condition and no copy, at which the
// compiler would wait for the stores too.
// The four waves of a narrow tile share its z: each adds every fourth range, and
// the four sums meet in LDS.
template <class D, int MT, int RK, bool BASE>
__global__ __launch_bounds__(256) void k_expand(AdapterParams p) {
  typedef typename D::vec vec;
  typedef typename D::elem elem;
  constexpr int NP = Parts<D>::N, kStep = MT == 4 ? 64 : 256;
  __shared__ TileLds tl;
  __shared__ __align__(16) float turn[4][16][64 + 4];
  __shared__ fx8 zs[MT == 1 ? 4 : 1][RK][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = lane & 15, g = lane >> 4;
  int a, rank;
  if (!find_tile<16 * MT>(p, blockIdx.x, tl, a, rank)) return;
  if (rank == 0 && p.base == p.out) return;
  const int first = tl.toks[MT == 4 ? 16 * wave : 0], mine = tl.toks[(MT == 4 ? 16 * wave : 0) + n];
  // Loads are unconditional, and a wide tile's stores: rows past the tile's end
  // repeat the wave's first token (and store its values again), ranks past the
  // adapter's its first 8.
  const int t = mine < 0 ? first : mine;
  const int c0 = blockIdx.y * p.cols + (MT == 4 ? 0 : 64 * wave);
  const int ce = (int)(blockIdx.y + 1) * p.cols, c1 = ce < p.N ? ce : p.N;
  if (MT == 4 && first < 0) return;  // this wave's rows are past the tile's end
  // rows of memory accesses: token 4 i + g, columns 4 n ..
  size_t row[4];
  unsigned live = 0;  // narrow tiles, mostly of a few tokens, store no row twice
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int u = tl.toks[(MT == 4 ? 16 * wave : 0) + 4 * i + g];
    row[i] = (size_t)(u < 0 ? first : u) * p.N + 4 * n;
    live |= (u < 0 ? 0u : 1u) << (4 * i);
  }
  if (rank == 0) {  // no adapter
    for (int c = c0; c < c1; c += kStep)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *(acc4*)(p.out + row[i] + c) = BASE ? *(const acc4*)(p.base + row[i] + c) : (acc4)(0.0f);
    return;
  }
  struct Cols {
    acc4 base[4];
    vec b[4][RK];
  };
  int kof[RK];
  ux4 mask[RK];  // clears B's columns past the rank, which hold anything
#pragma unroll
  for (int k = 0; k < RK; ++k) {
    kof[k] = 32 * k + 8 * g < rank ? 32 * k + 8 * g : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 32 * k + 8 * g + 2 * i;
      mask[k][i] = (r < rank ? 0xffffu : 0u) | (r + 1 < rank ? 0xffff0000u : 0u);
    }
  }
  const elem* brow = (const elem*)p.B + ((size_t)a * p.N + n) * p.R;
  const auto load = [&](int c, Cols& v) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v.base[j] = BASE ? stream_load((const acc4*)(p.base + row[j] + c)) : (acc4)(0.0f);
#pragma unroll
      for (int k = 0; k < RK; ++k) v.b[j][k] = *(const vec*)(brow + (size_t)(c + 16 * j) * p.R + kof[k]);
    }
  };
  Cols v0, v1;
  if (c0 < c1) load(c0, v0);
  const float scale = p.scales ? p.scales[a] : 1.0f;
  constexpr int kShare = MT == 1 ? 4 : 1;
  fx8 zv[RK];
#pragma unroll
  for (int k = 0; k < RK; ++k) {
    zv[k] = (fx8)(0.0f);
    const float* src = p.z + (size_t)t * p.R + kof[k];
#pragma unroll 4
    for (int s = MT == 1 ? wave : 0; s < p.ranges; s += kShare) zv[k] += load8(src + (size_t)s * p.T * p.R);
  }
  if (MT == 1) {
#pragma unroll
    for (int k = 0; k < RK; ++k) zs[wave][k][lane] = zv[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < RK; ++k) zv[k] = (zs[0][k][lane] + zs[1][k][lane]) + (zs[2][k][lane] + zs[3][k][lane]);
  }
  if (c0 >= c1) return;  // this wave's columns are past the end
  bx8 z[RK][3];
#pragma unroll
  for (int k = 0; k < RK; ++k) {
#pragma unroll
    for (int i = 0; i < 8; ++i) zv[k][i] = 32 * k + 8 * g + i < rank ? zv[k][i] * scale : 0.0f;
    cut<3>(zv[k], z[k]);
  }
  const auto work = [&](int c, const Cols& v) {
    acc4 d[4];
#pragma unroll
    for (int k = 0; k < RK; ++k) {
      bx8 q[4][NP];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        Parts<D>::of(__builtin_bit_cast(vec, __builtin_bit_cast(ux4, v.b[j][k]) & mask[k]), q[j]);
#pragma unroll
      for (int u = NP - 1; u >= 0; --u)
#pragma unroll
        for (int i = 2 - u; i >= 0; --i)
#pragma unroll
          for (int j = 0; j < 4; ++j) d[j] = mfma(q[j][u], z[k][i], k == 0 && u == NP - 1 && i == 2 - u ? (acc4)(0.0f) : d[j]);
    }
    // one wave's LDS accesses run in order
#pragma unroll
    for (int j = 0; j < 4; ++j) *(acc4*)&turn[wave][n][16 * j + 4 * g] = d[j];
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const acc4 sum = v.base[i] + *(const acc4*)&turn[wave][4 * i + g][4 * n];
      if (MT == 4 || live >> (4 * i) & 1) stream_store((acc4*)(p.out + row[i] + c), sum);
    }
    __builtin_amdgcn_wave_barrier();
  };
  const int last = c0 + (c1 - 1 - c0) / kStep * kStep;
  for (int c = c0;; c += 2 * kStep) {
    load(c + kStep < last ? c + kStep : last, v1);
    work(c, v0);
    if (c + kStep > last) break;
    load(c + 2 * kStep < last ? c + 2 * kStep : last, v0);
    work(c + kStep, v1);
    if (c + 2 * kStep > last) break;
  }
}

template <class D, int MT, bool BASE>
void expand(const AdapterParams& p, dim3 grid, hipStream_t s) {
  if (p.R <= 32) k_expand<D, MT, 1, BASE><<<grid, 256, 0, s>>>(p);
  else if (p.R <= 64) k_expand<D, MT, 2, BASE><<<grid, 256, 0, s>>>(p);
  else k_expand<D, MT, 4, BASE><<<grid, 256, 0, s>>>(p);
}

template <class D, int MT>
void shrink_expand(const AdapterParams& p, int tiles, hipStream_t s) {
  const dim3 gs(tiles, p.ranges), ge(tiles, (p.N + p.cols - 1) / p.cols);
  constexpr int kLeast = MT == 1 ? 1 : 2;  // wide tiles have ranks above 16
  if (p.R <= 16 * kLeast) k_shrink<D, MT, kLeast><<<gs, 64 * shrink_waves(MT), 0, s>>>(p);
  else if (p.R <= 32) k_shrink<D, MT, 2><<<gs, 64 * shrink_waves(MT), 0, s>>>(p);
  else if (p.R <= 64) k_shrink<D, MT, 4><<<gs, 64 * shrink_waves(MT), 0, s>>>(p);
  else k_shrink<D, MT, 8><<<gs, 64 * shrink_waves(MT), 0, s>>>(p);
  if (p.base) expand<D, MT, true>(p, ge, s);
  else expand<D, MT, false>(p, ge, s);
}

}  // namespace

AdapterWs adapter_ws(int T, int Kd, int n, int R) {
  AdapterWs w{};
  w.scan = T <= kAdapterScanT;
  // 64-token tiles, which read an adapter's weights a quarter as often, for ranks
  // above 16 where adapters hold 256 tokens or more on average. The whole call, us
  // with 16- and with 64-token tiles, ranks up to R, by tokens a group (of n + 1):
  //                            192       256       384       512       1024
  //   R 32, 4096^2,  4 groups  21/27     23/30     28/31     35/39     55/52
  //                 16         47/46     56/59     76/74     95/106    186/189
  //   R 64, 2816^2,  4         25/36     30/41     30/41     38/40     53/52
  //                 16         51/55     55/59     80/71     92/94     184/147
  //   R 128, 2816^2, 4         39/58     47/66     54/55     58/53     84/78
  //                 16         81/90     89/93     136/101   162/118   317/205
  // Below 256 16-token tiles win; from there to 512 it goes by the groups, and above
  // by the rank. Rank 16, 2048^2, 6600 tokens each: 331 against 354.
  w.mt = R > 16 && T / (n + 1) >= 256 ? 4 : 1;
  const int rows = 16 * w.mt;
  w.max_tiles = (n + 1 < T ? n + 1 : T) + T / rows;
  // ranges of Kd: about 512 workgroups of 4 waves, or 320 of 8 for wide tiles, at
  // least a step of 32 for each wave
  w.ranges = w.max_tiles > 0 ? (w.mt == 4 ? 320 : 512) / w.max_tiles : 1;
  if (w.ranges > Kd / 128) w.ranges = Kd / 128;
  if (w.ranges > 16) w.ranges = 16;
  if (w.ranges < 1) w.ranges = 1;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) & ~(size_t)255;
    return at;
  };
  w.z = take((size_t)w.ranges * T * R * 4);
  w.perm = take(w.scan ? 0 : (size_t)w.max_tiles * rows * 4);
  w.tiles = take(w.scan ? 0 : ((size_t)w.max_tiles * 2 + 4) * 4);
  w.total = off < 256 ? 256 : off;
  return w;
}

hipError_t launch_adapters(const AdapterParams& q, const AdapterWs& w, bool bf16, hipStream_t s) {
  AdapterParams p = q;
  // columns of an expand workgroup: 512 of a wide tile; of a narrow one up to 1024
  // (4093 x 2816: 33.8 us against 36.2 with 512), fewer where that makes less than
  // 512 workgroups (128 tokens of 64 adapters: 7.3 against 8.8)
  p.cols = w.mt == 4 ? 512 : 1024;
  while (w.mt == 1 && p.cols > 256 && (long long)w.max_tiles * ((p.N + p.cols - 1) / p.cols) < 512) p.cols /= 2;
  if (!w.scan) k_plan<<<1, 1024, 0, s>>>(p, 16 * w.mt);
  if (bf16) {
    if (w.mt == 4) shrink_expand<BF16, 4>(p, w.max_tiles, s);
    else shrink_expand<BF16, 1>(p, w.max_tiles, s);
  } else {
    if (w.mt == 4) shrink_expand<F16, 4>(p, w.max_tiles, s);
    else shrink_expand<F16, 1>(p, w.max_tiles, s);
  }
  return hipGetLastError();
}

}  // namespace mpb
