// Grouping of rows by key, and the embedding table's lookup and gradient.
//
// Grouping is a stable counting sort: position of row i = rows of smaller keys + rows
// before i of the same key.  Up to GROUP_ONE rows one launch does it in LDS; beyond,
// every digit of the key takes two launches (count per block, move; three from 524289
// rows on).  A key outside [0, num_keys) counts as num_keys: its rows come last.
// Counts and ranks are integers, so the result is exact and the same every time.
// Bound by launches: 256 rows 7.6 us (a launch alone takes 3.6), 524288 rows with one
// digit 13.8 us, of which the count takes 3 and the move, on half of the compute units, 12.
// 9000 and 100000 rows over 50000 keys, five launches: 28 and 31 us.  524289 rows with one
// digit, three launches, 18.7 us; 2000000 rows 45 us, over 50000 keys 110 us.
//
// The embedding's two calls are bound by HBM: 65536 rows of a 131072 x 4096 bf16 table,
// 136 us for the lookup (5.2 TB/s) and 370 us for the gradient: 35 us of grouping, 315 us
// for the sums and zeros (5.2 TB/s), 24 us for tokens that cross chunks.
#pragma once

#include "common.h"

namespace mo {

constexpr int GROUP_ONE = 8192;      // rows that one block sorts in LDS
constexpr int GROUP_ROUNDS = 4;            // times 1024: rows of a block beyond that
constexpr int GROUP_BITS = 9;        // most bits of a digit (kernels for 4, 7, 8 and 9)
constexpr int GROUP_DIGITS = 1 << GROUP_BITS;

struct KeySource {
  const void* keys;   // int32 or int64
  int is64;
  uint32_t num_keys;
};

__device__ inline uint32_t load_key(const KeySource& s, int64_t i) {
  if (s.is64) {
    const int64_t k = static_cast<const int64_t*>(s.keys)[i];
    return (k >= 0 && k < static_cast<int64_t>(s.num_keys)) ? static_cast<uint32_t>(k) : s.num_keys;
  }
  const int32_t k = static_cast<const int32_t*>(s.keys)[i];
  return (k >= 0 && static_cast<uint32_t>(k) < s.num_keys) ? static_cast<uint32_t>(k) : s.num_keys;
}

// Rank of this lane's digit among the wave's earlier elements, whose counts so far are
// in hist[digit * STRIDE] (this wave's); adds the wave's 64 elements to it.
template <int STRIDE, int BITS>
__device__ inline uint32_t wave_rank(uint32_t* hist, uint32_t d, bool live) {
  uint64_t peers = __ballot(live);
#pragma unroll
  for (int b = 0; b < BITS; ++b) {
    const uint64_t m = __ballot((d >> b) & 1);
    peers &= ((d >> b) & 1) ? m : ~m;
  }
  const uint64_t below = (uint64_t(1) << (threadIdx.x & 63)) - 1;
  uint32_t rank = 0;
  if (live) {
    const uint32_t before = hist[d * STRIDE];
    rank = before + __popcll(peers & below);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if ((peers & below) == 0) hist[d * STRIDE] = before + __popcll(peers);   // the first of its peers
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  return rank;
}

// Exclusive running sum of v[0..count) over a block of NT threads, in place, each thread
// a run of consecutive words.  scratch: NT / 64 words.
template <int NT>
__device__ inline void block_scan(uint32_t* v, int count, uint32_t* scratch) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int per = (count + NT - 1) / NT, lo = min(count, tid * per), hi = min(count, lo + per);
  uint32_t own = 0;
  for (int i = lo; i < hi; ++i) own += v[i];
  uint32_t inc = own;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t up = __shfl_up(inc, d);
    if (lane >= d) inc += up;
  }
  if (lane == 63) scratch[wave] = inc;
  __syncthreads();
  uint32_t run = inc - own;
#pragma unroll
  for (int w = 0; w < NT / 64; ++w) run += w < wave ? scratch[w] : 0;
  for (int i = lo; i < hi; ++i) {
    const uint32_t x = v[i];
    v[i] = run;
    run += x;
  }
  __syncthreads();
}

// Zeros over memory that starts at any element of 2 or 4 bytes, 256 KiB a block.
struct ZeroFill {
  void* p;
  int64_t bytes;     // 0: nothing to fill
};
constexpr int64_t ZERO_BLOCK = 256 * 1024;
__device__ inline void zero_fill(const ZeroFill& z, int64_t block) {
  typedef u32x4_t any_t __attribute__((aligned(2)));
  typedef __attribute__((address_space(1))) unsigned char* bytes_t;
  const u32x4_t v = {0, 0, 0, 0};
  const bytes_t p = (bytes_t)static_cast<unsigned char*>(z.p) + block * ZERO_BLOCK;
  const int count = static_cast<int>(min(z.bytes - block * ZERO_BLOCK, ZERO_BLOCK));
  const int whole = count & ~15;
  for (int i = threadIdx.x * 16; i < whole; i += 1024 * 16)
    __builtin_nontemporal_store(v, reinterpret_cast<gptr<any_t>>(p + i));
  const int i = whole + threadIdx.x * 2;
  if (i < count) *reinterpret_cast<gptr<uint16_t>>(p + i) = 0;
}

// ---- up to GROUP_ONE rows: every one of `sorters` blocks sorts them all in LDS; block 0
// writes the order, and the sorters share the offsets (binary searches in the sorted
// keys).  The sort leaves the device nearly idle, so the blocks behind clear the memory
// that the caller's next launch adds rows to.
template <int BITS>
__global__ __launch_bounds__(1024) void k_group_small(KeySource src, int n, int passes, int sorters, ZeroFill zero,
                                                      int32_t* __restrict__ order, int32_t* __restrict__ offsets) {
  if (static_cast<int>(blockIdx.x) >= sorters) {
    zero_fill(zero, static_cast<int>(blockIdx.x) - sorters);
    return;
  }
  __shared__ uint32_t key[2][GROUP_ONE];
  __shared__ uint16_t row[2][GROUP_ONE];
  // [digit][wave]: one running sum gives all positions.  17 words a digit (the last
  // stays 0), so that digits do not share banks.
  constexpr int HP = 17;
  __shared__ uint32_t hist[GROUP_DIGITS * HP];
  __shared__ uint32_t scratch[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int per = (n + 1023) / 1024;             // rounds of 64 per wave
  for (int i = tid; i < n; i += 1024) {
    key[0][i] = load_key(src, i);
    row[0][i] = static_cast<uint16_t>(i);
  }
  constexpr int bits = BITS, nd = 1 << BITS;
  int from = 0;
  for (int p = 0; p < passes; ++p) {
    for (int i = tid; i < nd * HP; i += 1024) hist[i] = 0;
    __syncthreads();
    uint32_t rank[GROUP_ONE / 1024];
    const uint32_t mask = nd - 1;
#pragma unroll
    for (int r = 0; r < GROUP_ONE / 1024; ++r) {
      if (r >= per) break;
      const int i = wave * per * 64 + r * 64 + lane;
      const bool live = i < n;
      const uint32_t d = live ? (key[from][i] >> (p * bits)) & mask : 0;
      rank[r] = wave_rank<HP, BITS>(hist + wave, d, live);
    }
    __syncthreads();
    block_scan<1024>(hist, nd * HP, scratch);
#pragma unroll
    for (int r = 0; r < GROUP_ONE / 1024; ++r) {
      if (r >= per) break;
      const int i = wave * per * 64 + r * 64 + lane;
      if (i < n) {
        const uint32_t k = key[from][i];
        const uint32_t pos = hist[((k >> (p * bits)) & mask) * HP + wave] + rank[r];
        key[from ^ 1][pos] = k;
        row[from ^ 1][pos] = row[from][i];
      }
    }
    from ^= 1;
    __syncthreads();
  }
  if (blockIdx.x == 0)
    for (int i = tid; i < n; i += 1024) order[i] = row[from][i];
  const int64_t count = static_cast<int64_t>(src.num_keys) + 1;
  const int64_t step = static_cast<int64_t>(sorters) * 1024;
  for (int64_t v = static_cast<int64_t>(blockIdx.x) * 1024 + tid; v < count; v += step) {
    int lo = 0, hi = n;   // first position whose key is at least v
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (key[from][mid] < v) lo = mid + 1; else hi = mid;
    }
    offsets[v] = lo;
  }
}

// ---- any number of rows, one digit: counts[block][digit].  A block of 1024 threads has
// 4096 rows, its wave w the 256 rows from 256 w on.
template <bool FIRST>
__global__ __launch_bounds__(1024) void k_group_count(KeySource src, const uint2* __restrict__ pairs, int64_t n,
                                                      int shift, int bits, uint32_t* __restrict__ counts) {
  __shared__ uint32_t h[GROUP_DIGITS];
  const int nd = 1 << bits;
  for (int i = threadIdx.x; i < nd; i += 1024) h[i] = 0;
  __syncthreads();
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (GROUP_ROUNDS * 1024);
#pragma unroll
  for (int r = 0; r < GROUP_ROUNDS; ++r) {
    const int64_t i = i0 + r * 1024 + threadIdx.x;
    if (i < n) {
      const uint32_t k = FIRST ? load_key(src, i) : pairs[i].x;
      atomicAdd(&h[(k >> shift) & (nd - 1)], 1u);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < nd; i += 1024) counts[static_cast<int64_t>(blockIdx.x) * nd + i] = h[i];
}

// Beyond GROUP_SUMS blocks: every digit's counts become running sums over the blocks,
// and totals[digit].  One thread per digit.
constexpr int GROUP_SUMS = 128;
__global__ __launch_bounds__(64) void k_group_scan(uint32_t* __restrict__ counts, int nblk, int nd,
                                                   uint32_t* __restrict__ totals) {
  const int d = blockIdx.x * 64 + threadIdx.x;
  if (d >= nd) return;
  uint32_t run = 0;
  constexpr int B = 16;
  for (int b0 = 0; b0 < nblk; b0 += B) {
    uint32_t x[B];
#pragma unroll
    for (int u = 0; u < B; ++u) x[u] = counts[static_cast<int64_t>(min(b0 + u, nblk - 1)) * nd + d];
#pragma unroll
    for (int u = 0; u < B; ++u) {
      if (b0 + u >= nblk) break;
      counts[static_cast<int64_t>(b0 + u) * nd + d] = run;
      run += x[u];
    }
  }
  totals[d] = run;
}

// Moves every row to its place: rows of smaller digits + this digit's rows in earlier
// blocks + in earlier waves + in earlier lanes.  Up to GROUP_SUMS blocks, each adds the
// earlier blocks' counts itself (a launch less: 4 us); beyond, totals are given.  The
// last digit's pass writes the order; the keys go along where another pass or the
// search for the offsets reads them.  With a single digit its running sums are the
// offsets.
template <int BITS, bool FIRST, bool LAST>
__global__ __launch_bounds__(1024) void k_group_move(KeySource src, const uint2* __restrict__ pairs, int64_t n,
                                                     int shift, int nblk, const uint32_t* __restrict__ counts,
                                                     const uint32_t* __restrict__ totals, uint2* __restrict__ out,
                                                     uint32_t* __restrict__ keys_out, int32_t* __restrict__ order,
                                                     int32_t* __restrict__ offsets) {
  constexpr int nd = 1 << BITS;
  constexpr int PARTS = 1024 / nd;        // threads per digit for the sums over blocks
  __shared__ uint32_t base[nd], mine[nd];
  __shared__ uint32_t wh[16][nd];
  __shared__ uint32_t scratch[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (GROUP_ROUNDS * 1024) + wave * (GROUP_ROUNDS * 64) + lane;
  uint32_t rank[GROUP_ROUNDS], k[GROUP_ROUNDS], at[GROUP_ROUNDS];
#pragma unroll
  for (int r = 0; r < GROUP_ROUNDS; ++r) {
    const int64_t i = i0 + r * 64;
    k[r] = 0;
    at[r] = static_cast<uint32_t>(i);
    if (i < n) {
      if (FIRST) {
        k[r] = load_key(src, i);
      } else {
        const uint2 p = pairs[i];
        k[r] = p.x;
        at[r] = p.y;
      }
    }
  }
  for (int i = tid; i < 16 * nd; i += 1024) wh[i / nd][i % nd] = 0;
  if (totals) {
    for (int i = tid; i < nd; i += 1024) {
      base[i] = totals[i];
      mine[i] = counts[static_cast<int64_t>(blockIdx.x) * nd + i];
    }
    __syncthreads();
  } else {
    for (int i = tid; i < nd; i += 1024) base[i] = mine[i] = 0;
    __syncthreads();
    const int d = tid % nd, part = tid / nd;
    const int per = (nblk + PARTS - 1) / PARTS;
    uint32_t all = 0, before = 0;
    constexpr int B = 16;
    for (int u0 = 0; u0 < per; u0 += B) {
      uint32_t x[B];
#pragma unroll
      for (int u = 0; u < B; ++u) x[u] = counts[min(part * per + u0 + u, nblk - 1) * nd + d];
#pragma unroll
      for (int u = 0; u < B; ++u) {
        const int b = part * per + u0 + u;
        const bool mine_too = u0 + u < per && b < nblk;
        all += mine_too ? x[u] : 0;
        before += mine_too && b < static_cast<int>(blockIdx.x) ? x[u] : 0;
      }
    }
    atomicAdd(&base[d], all);
    atomicAdd(&mine[d], before);
    __syncthreads();
  }
  block_scan<1024>(base, nd, scratch);
  if (FIRST && LAST && blockIdx.x == 0)
    for (int i = tid; i <= static_cast<int>(src.num_keys); i += 1024) offsets[i] = static_cast<int32_t>(base[i]);
#pragma unroll
  for (int r = 0; r < GROUP_ROUNDS; ++r)
    rank[r] = wave_rank<1, BITS>(wh[wave], (k[r] >> shift) & (nd - 1), i0 + r * 64 < n);
  __syncthreads();
  for (int i = tid; i < nd; i += 1024) {
    uint32_t run = base[i] + mine[i];
#pragma unroll
    for (int w = 0; w < 16; ++w) {
      const uint32_t c = wh[w][i];
      wh[w][i] = run;
      run += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < GROUP_ROUNDS; ++r) {
    if (i0 + r * 64 >= n) continue;
    const uint32_t pos = wh[wave][(k[r] >> shift) & (nd - 1)] + rank[r];
    if (LAST) {
      order[pos] = static_cast<int32_t>(at[r]);
      if (!FIRST) keys_out[pos] = k[r];
    } else {
      out[pos] = make_uint2(k[r], at[r]);
    }
  }
}

// offsets[v] = first position whose key is at least v
__global__ __launch_bounds__(256) void k_group_offsets(const uint32_t* __restrict__ keys, int64_t n, int64_t count,
                                                       int32_t* __restrict__ offsets) {
  const int64_t v = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (v >= count) return;
  int64_t lo = 0, hi = n;
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (keys[mid] < v) lo = mid + 1; else hi = mid;
  }
  offsets[v] = static_cast<int32_t>(lo);
}

__global__ __launch_bounds__(256) void k_group_none(int32_t* __restrict__ offsets, int64_t count) {
  const int64_t v = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (v < count) offsets[v] = 0;
}

// ---------------------------------------------------------------- rows of values

// A lane's share of a row: ROW_W consecutive values from column c on, moved 16 bytes at
// a time with the element's alignment (rows may start anywhere).  The share that would
// pass the row's end starts at width - ROW_W instead: its first values are a neighbour's
// too, and both compute and store the same.  So no lane branches and loads can be kept
// in flight.  Only rows shorter than ROW_W (WIDE false) go element by element.
constexpr int ROW_W = 8;
typedef u32x4_t u32x4_any2 __attribute__((aligned(2)));
typedef u32x4_t u32x4_any4 __attribute__((aligned(4)));
template <typename T> struct Any16 { typedef u32x4_any4 type; };
template <> struct Any16<bf16_t> { typedef u32x4_any2 type; };

template <bool WIDE>
__device__ inline int share_at(int c, int width) { return WIDE ? min(c, width - ROW_W) : c; }

template <typename T, bool WIDE>
struct Share {
  static constexpr int N = 16 / sizeof(T);
  typedef T vt __attribute__((ext_vector_type(N)));
  u32x4_t w[ROW_W / N];
  __device__ inline void load(const T* row, int c, int width) {
    if constexpr (WIDE) {
#pragma unroll
      for (int p = 0; p < ROW_W / N; ++p)
        w[p] = *reinterpret_cast<gptr<const typename Any16<T>::type>>(global(row + c + p * N));
    } else {
      vt x[ROW_W / N];
#pragma unroll
      for (int i = 0; i < ROW_W; ++i) x[i / N][i % N] = c + i < width ? global(row)[c + i] : from_f32<T>(0.f);
#pragma unroll
      for (int p = 0; p < ROW_W / N; ++p) w[p] = __builtin_bit_cast(u32x4_t, x[p]);
    }
  }
  __device__ inline void values(float (&v)[ROW_W]) const {
#pragma unroll
    for (int p = 0; p < ROW_W / N; ++p) {
      const vt x = __builtin_bit_cast(vt, w[p]);
#pragma unroll
      for (int i = 0; i < N; ++i) v[p * N + i] = to_f32(x[i]);
    }
  }
};
// bf16: consecutive lanes write consecutive 16 bytes, whole lines that nobody reads
// soon, so they pass the caches by.  fp32: a lane's 32 bytes take two instructions,
// which only the L2 joins to lines.
template <bool WIDE, typename T>
__device__ inline void store_w(T* row, int c, int width, const float (&v)[ROW_W]) {
  if constexpr (WIDE) {
    constexpr int N = 16 / sizeof(T);
    typedef T vt __attribute__((ext_vector_type(N)));
#pragma unroll
    for (int p = 0; p < ROW_W / N; ++p) {
      vt x;
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = from_f32<T>(v[p * N + i]);
      const u32x4_t w = __builtin_bit_cast(u32x4_t, x);
      const auto to = reinterpret_cast<gptr<typename Any16<T>::type>>(global(row + c + p * N));
      if constexpr (sizeof(T) == 2)
        __builtin_nontemporal_store(w, to);
      else
        *to = w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < ROW_W; ++i)
      if (c + i < width) global(row)[c + i] = from_f32<T>(v[i]);
  }
}
// zeros over one row by a block of NT threads
template <int NT, typename T>
__device__ inline void zero_row(T* row, int width) {
  constexpr int N = 16 / sizeof(T);
  const u32x4_t z = {0, 0, 0, 0};
  const int whole = width / N;
  for (int p = threadIdx.x; p < whole; p += NT)
    __builtin_nontemporal_store(z, reinterpret_cast<gptr<typename Any16<T>::type>>(global(row + p * N)));
  const int c = whole * N + threadIdx.x;
  if (c < width) global(row)[c] = from_f32<T>(0.f);
}

// out[i] = table[token[i]] * scale (fp32, rounded once); zeros for a token outside the
// table.  One wave per row.
template <typename T, typename TO, bool WIDE>
__global__ __launch_bounds__(256) void k_embed_lookup(const T* __restrict__ table, int64_t ldt, KeySource tokens,
                                                      int64_t first_block, int64_t n, int dim, float scale,
                                                      TO* __restrict__ out) {
  const int lane = threadIdx.x & 63;
  const int64_t i = (first_block + blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (i >= n) return;
  const uint32_t tok = __builtin_amdgcn_readfirstlane(load_key(tokens, i));
  TO* o = out + i * dim;
  const T* row = table + static_cast<int64_t>(tok) * ldt;
  const bool used = tok < tokens.num_keys;
  constexpr int U = 4;   // pieces of 512 values in flight (2: the same time)
  for (int c0 = 0; c0 < dim; c0 += U * 64 * ROW_W) {
    Share<T, WIDE> sh[U];
    if (used) {
#pragma unroll
      for (int u = 0; u < U; ++u) sh[u].load(row, share_at<WIDE>(c0 + (u * 64 + lane) * ROW_W, dim), dim);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + (u * 64 + lane) * ROW_W;
      float v[ROW_W] = {};
      if (used) {
        sh[u].values(v);
#pragma unroll
        for (int e = 0; e < ROW_W; ++e) v[e] *= scale;
      }
      if (c < dim) store_w<WIDE>(o, share_at<WIDE>(c, dim), dim, v);
    }
  }
}

// ---- gradient of the table: grad[v] = scale * sum of grad_out over the rows of token v.
//
// The rows in token order are cut into chunks of EG_ROWS positions.  A wave takes one
// chunk and 512 columns, adds the rows of a token in fp32 in the order of their
// positions, and stores a token that lies within the chunk.  A token that crosses
// chunks leaves fp32 partial sums (a chunk has one at its head and one at its tail at
// most), which a second launch adds in order: the sums do not depend on timing, and a
// token that holds a large share of all rows is spread over the device.  Tokens
// without rows are zeroed by the first launch's other blocks; up to GROUP_ONE rows the
// grouping's launch has zeroed the whole table by then (4099 rows of a 50001 x 2048 fp32
// table: 89 us; 97 us with the sort's 14 us and the filling one after the other).
constexpr int EG_ROWS = 32;
constexpr int EG_COLS = 64 * ROW_W;
constexpr int EG_ZERO = 8;     // table rows per zeroing block

struct EmbedGrad {
  const void* g;           // n x dim
  int64_t ldg;
  const int32_t* order;    // rows in token order
  const int32_t* offsets;  // vocab + 1
  KeySource tokens;
  int64_t n;
  int dim, parts;          // column parts of EG_COLS
  float scale;
  void* out;               // vocab x dim
  float* partial;          // [chunk][head, tail][pitch]
  int pitch;               // dim rounded up to a multiple of 8
  int32_t* tail_to;        // [chunk]: the last chunk of the token that crosses its end, -1: none
  int64_t run_blocks;
  int64_t first_block;     // of this launch
};

template <typename T, typename TO, bool WIDE>
__global__ __launch_bounds__(256) void k_embed_grad(EmbedGrad a) {
  const int lane = threadIdx.x & 63;
  const int64_t block = a.first_block + blockIdx.x;
  if (block >= a.run_blocks) {
    // zeros for tokens without rows: the block's threads run along the table row
    const int64_t v0 = (block - a.run_blocks) * EG_ZERO;
#pragma unroll
    for (int r = 0; r < EG_ZERO; ++r) {
      const int64_t v = v0 + r;
      if (v >= a.tokens.num_keys) return;
      if (a.offsets[v] != a.offsets[v + 1]) continue;
      zero_row<256>(static_cast<TO*>(a.out) + v * a.dim, a.dim);
    }
    return;
  }
  const int64_t item = block * 4 + (threadIdx.x >> 6);
  const int64_t kept = a.offsets[a.tokens.num_keys];
  const int64_t chunk = item / a.parts, p0 = chunk * EG_ROWS;
  const bool tells = lane == 0 && item % a.parts == 0 && p0 < a.n;   // for its chunk, once
  if (p0 >= kept) {
    if (tells) a.tail_to[chunk] = -1;
    return;
  }
  const int c0 = static_cast<int>(item % a.parts) * EG_COLS + lane * ROW_W, c = share_at<WIDE>(c0, a.dim);
  const int count = static_cast<int>(min(static_cast<int64_t>(EG_ROWS), kept - p0));
  // lane l: position p0 - 1 + l (its row and token), l <= count + 1; ~0: none
  int my_row = 0;
  uint32_t my_tok = ~0u;
  const int64_t p = p0 - 1 + lane;
  if (lane <= EG_ROWS + 1 && p >= 0 && p < kept) {
    my_row = a.order[p];
    my_tok = load_key(a.tokens, my_row);
  }
  const uint32_t before = __builtin_amdgcn_readlane(my_tok, 0);
  const uint32_t after = __builtin_amdgcn_readlane(my_tok, EG_ROWS + 1);
  uint32_t cur = __builtin_amdgcn_readlane(my_tok, 1);
  bool head = cur == before;   // the run at hand began in an earlier chunk
  float acc[ROW_W];
#pragma unroll
  for (int e = 0; e < ROW_W; ++e) acc[e] = 0.f;
  auto flush = [&](bool tail) {
    if (c0 >= a.dim) return;
    if (head || tail) {
      // c and the pitch need not be whole pieces: the partial sums are in fp32 rows
      float* q = a.partial + (chunk * 2 + (head ? 0 : 1)) * a.pitch;
      store_w<true>(q, c, a.pitch, acc);
    } else {
      float s[ROW_W];
#pragma unroll
      for (int e = 0; e < ROW_W; ++e) s[e] = acc[e] * a.scale;
      store_w<WIDE>(static_cast<TO*>(a.out) + static_cast<int64_t>(cur) * a.dim, c, a.dim, s);
    }
  };
  constexpr int B = 8;   // rows in flight
  for (int r0 = 0; r0 < count; r0 += B) {
    Share<T, WIDE> sh[B];
#pragma unroll
    for (int u = 0; u < B; ++u) {   // past the last row: the last row again
      const int64_t row = __builtin_amdgcn_readlane(my_row, min(r0 + u, count - 1) + 1);
      sh[u].load(static_cast<const T*>(a.g) + row * a.ldg, c, a.dim);
    }
#pragma unroll
    for (int u = 0; u < B; ++u) {
      if (r0 + u >= count) break;
      const uint32_t t = __builtin_amdgcn_readlane(my_tok, r0 + u + 1);
      if (t != cur) {
        flush(false);
        cur = t;
        head = false;
#pragma unroll
        for (int e = 0; e < ROW_W; ++e) acc[e] = 0.f;
      }
      float v[ROW_W];
      sh[u].values(v);
#pragma unroll
      for (int e = 0; e < ROW_W; ++e) acc[e] += v[e];
    }
  }
  const bool crosses = count == EG_ROWS && cur == after;
  flush(crosses);
  if (tells) a.tail_to[chunk] = crosses && !head ? (a.offsets[cur + 1] - 1) / EG_ROWS : -1;
}

// Tokens that cross chunks: the tail of the chunk where the token begins, then the
// heads of the following chunks.  A block looks through 8 chunks for 256 columns and
// deals those that have such a token to its waves; a wave keeps 32 partial sums in
// flight, since a token that holds 8% of 65536 rows has 174 of them.  (A wave per chunk
// that finds out for itself: 49 us, nearly all of it waves that find nothing; 24 us so.)
constexpr int EJ_COLS = 64 * 4, EJ_CHUNKS = 8;
template <typename TO>
__device__ inline void join_token(const EmbedGrad& a, int64_t chunk, int64_t to, int c) {
  const uint32_t tok = load_key(a.tokens, a.order[chunk * EG_ROWS + EG_ROWS - 1]);
  if (c >= a.dim) return;
  const int have = min(4, a.dim - c);
  auto part = [&](int64_t q, int which) {   // the pitch has room for whole pieces
    return *reinterpret_cast<gptr<const f32x4_t>>(global(a.partial + (q * 2 + which) * a.pitch + c));
  };
  f32x4_t s = part(chunk, 1);
  constexpr int B = 32;
  for (int64_t q0 = chunk + 1; q0 <= to; q0 += B) {
    f32x4_t v[B];
#pragma unroll
    for (int u = 0; u < B; ++u) v[u] = part(min(q0 + u, to), 0);   // no lane branches
#pragma unroll
    for (int u = 0; u < B; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] += q0 + u <= to ? v[u][e] : 0.f;
  }
  TO* o = static_cast<TO*>(a.out) + static_cast<int64_t>(tok) * a.dim + c;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < have) global(o)[e] = from_f32<TO>(s[e] * a.scale);
}

template <typename TO>
__global__ __launch_bounds__(256) void k_embed_join(EmbedGrad a, int parts) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t first = static_cast<int64_t>(blockIdx.x / parts) * EJ_CHUNKS, chunks = (a.n + EG_ROWS - 1) / EG_ROWS;
  const int c = static_cast<int>(blockIdx.x % parts) * EJ_COLS + lane * 4;
  const int to = lane < EJ_CHUNKS && first + lane < chunks ? a.tail_to[first + lane] : -1;
  int nth = 0;
  for (uint64_t left = __ballot(to >= 0); left != 0; left &= left - 1, ++nth) {
    const int at = __ffsll(static_cast<unsigned long long>(left)) - 1;
    if ((nth & 3) == wave) join_token<TO>(a, first + at, __builtin_amdgcn_readlane(to, at), c);
  }
}

}  // namespace mo
