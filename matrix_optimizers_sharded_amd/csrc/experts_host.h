// Host side of the grouped products: argument checks, the choice of a tile and the
// launch.  One translation unit per product instantiates it (expert_*.hip).
#pragma once

#include <algorithm>

#include "experts.h"
#include "host.h"

namespace mo {

struct XCall {
  XArgs a;
  int dtype, out;
  bool p_direct, q_direct;   // operands whose rows all start and end on 16 bytes
};

inline int check_expert(const char* pa, const void* A, int64_t lda, int64_t wa, const char* pb, const void* B,
                        int64_t ldb, int64_t wb, const int32_t* offsets, int32_t experts, int64_t n, int64_t k,
                        int64_t m, int32_t dtype, int32_t out_dtype, const void* C) {
  if (!valid_dtype(dtype) || !valid_dtype(out_dtype))
    return fail(MO_ERR_UNSUPPORTED, "dtypes must be MO_F32 or MO_BF16");
  if (dtype == MO_F32 && out_dtype != MO_F32)
    return fail(MO_ERR_UNSUPPORTED, "fp32 operands give fp32 results");
  if (experts < 1 || experts > X_MAX_EXPERTS)
    return fail(MO_ERR_INVALID, "experts must be in [1, " + std::to_string(X_MAX_EXPERTS) + "]");
  // rounded up to whole tiles and slabs, a segment's rows still fit 32 bits
  if (n < 0 || n > 0x7fffffffLL - 1023) return fail(MO_ERR_INVALID, "n must be in [0, 2^31 - 1024]");
  constexpr int64_t MAXW = int64_t(1) << 20;
  if (k < 1 || m < 1 || k > MAXW || m > MAXW) return fail(MO_ERR_INVALID, "k and m must be in [1, 2^20]");
  if (lda < wa || lda > MAXW) return fail(MO_ERR_INVALID, std::string(pa) + ": the row pitch must be in [width, 2^20]");
  if (ldb < wb || ldb > MAXW) return fail(MO_ERR_INVALID, std::string(pb) + ": the row pitch must be in [width, 2^20]");
  if (!offsets) return fail(MO_ERR_INVALID, "offsets is NULL");
  if (n > 0 && !C) return fail(MO_ERR_INVALID, "the result is NULL");
  if (n > 0 && (!A || !B)) return fail(MO_ERR_INVALID, std::string(pa) + " or " + pb + " is NULL");
  return MO_OK;
}

// The result, `rows` x `width`, and the operands' rows.
inline int check_result(const void* C, int64_t rows, int64_t width, int32_t out_dtype, const ByteRows& a,
                        const ByteRows& b, const int32_t* offsets, int32_t experts) {
  return check_apart("the result", byte_rows(C, rows, width, width, dtype_size(out_dtype)),
                     {a, b, byte_rows(offsets, 1, experts + 1, experts + 1, 4)});
}

// An operand that can be loaded straight into LDS: rows of `width` elements, `pitch` apart.
inline bool direct_rows(const void* p, int64_t pitch, int64_t width, int64_t es) {
  return aligned16(p) && pitch * es % 16 == 0 && width * es % 16 == 0;
}

// Row tiles of T rows that n rows in `experts` segments can make, at most (the rows of
// no segment make two more pieces).
inline int64_t row_tiles(int64_t n, int experts, int T) { return n / T + experts + 2; }

template <int KIND, int TM, int TN>
int64_t most_tiles(const XArgs& a) {
  if (KIND == X_DW) return cdiv(a.m, TM) * cdiv(a.k, TN) * a.experts;
  return std::min<int64_t>(a.n, row_tiles(a.n, a.experts, TM)) * cdiv(KIND == X_FWD ? a.m : a.k, TN);
}

template <typename T, int KIND, typename TO, int TM, int TN, int WR, int WC, int STAGES, int LOAD>
int launch_tile(int pk, XArgs a, hipStream_t stream) {
  typedef XGemm<T, KIND, TM, TN, WR, WC, STAGES, TO, LOAD> G;
  constexpr int LDS_PER_CU = 160 * 1024;
  a.slots = device_cus() * std::max(1, LDS_PER_CU / XLds<G>::bytes);
  const int64_t tiles = most_tiles<KIND, TM, TN>(a);
  if (tiles == 0) return MO_OK;
  const int64_t blocks = x_blocks(tiles, G::SPLITS, a.slots);
  if (blocks > 0x7fffffffLL) return fail(MO_ERR_INVALID, "too many tiles");
  return launch_blocks(pk, stream, blocks, G::NT, [&](int64_t first, uint32_t count) {
    a.first_block = first;
    hipLaunchKernelGGL((k_expert<G, KIND>), dim3(count), dim3(G::NT), 0, stream, a);
  });
}

template <typename T, int KIND, typename TO, int LOAD>
int launch_split(int pk, XArgs a, hipStream_t stream) {
  typedef XSplit<T, KIND, TO, LOAD, 4> G;
  const int64_t tiles = most_tiles<KIND, G::TM, G::TN>(a);
  if (tiles > 0x7fffffffLL) return fail(MO_ERR_INVALID, "too many tiles");
  return launch_blocks(pk, stream, tiles, G::NT, [&](int64_t first, uint32_t count) {
    a.first_block = first;
    hipLaunchKernelGGL((k_expert_split<G, KIND>), dim3(count), dim3(G::NT), 0, stream, a);
  });
}

// Which kernel and tile.  A large tile reads its operands fewer times, a small one keeps
// more compute units busy.  The segments' sizes are on the device, so the choice sees the
// mean rows of an expert, idle experts among them.  Times in us for forward / input
// gradient, operands in the caches where they fit, the other choice in brackets.
// 1. Few rows per expert, or few tiles, and a sum of four slabs or more: four waves split
//    the sum (64 x 64 tiles in brackets).  One row: 7.7 (15) / 13 (35).  16 experts, 2048 x
//    2816, bf16: 32 rows each 30 (31) / 33 (34), 33 rows 36 (31) / 36 (34); fp32, 1024 x 2048: 32
//    rows 27 (44) / 27 (54), 33 rows 45 (43) / 43 (54).  Few tiles: 1001 rows over 6
//    experts, 768 x 1000, fp32: 26 (33) / 24 (29); 1024 rows, one expert, 2048 x 2048, two
//    tiles a compute unit, fp32: 78 (80) / 78 (81), but bf16 25 (21) / 23 (20).  A sum of four
//    slabs, 128 rows, 16 experts, 256 x 2816: 6.8 (7.1).
//    Weight gradients: 2 experts of 1024 rows, bf16: 768 x 640, 240 tiles, 7.3 (8.4); 768 x
//    768, 288 tiles, split 9.3, 64 x 64 10.1.  16384 rows, 512 x 768, 2 experts: 35 (52).
//    Eight waves were faster only for a single expert's 128 x 128 gradient: 36 (41).
// 2. Weight gradients with sums of one or two slabs are all stores: one slab in LDS, so
//    that four blocks share a compute unit.  300 rows over 128 experts, 1024 x 2048: 100
//    (122, two slabs).  64 experts of 128 rows: 72 (92; 256 x 256: 77), of 129: 86 (256 x 256: 86).
// 3. bf16, segments of 160 rows or more: 256 x 256 (128 x 128 in brackets).  16384 rows, 8
//    experts, 4096 x 11008: 1290 (1640) / 1310 (1680), weight gradient 1300 (1710).  32
//    experts, 2048 x 2816: 96 rows each 100 (102) / 71 (75), 159 rows 110 (121) / 92 (117), 160
//    rows 110 (125) / 92 (120), 320 rows 181 (167) / 174 (175).  With odd widths, through
//    registers, 8192 rows, 4 experts, 4095 x 5631: 450 / 500 / 505.
// 4. 128 x 128, or 64 x 64 where there would be fewer tiles than compute units (in
//    brackets).  64 experts, 2048 x 1408, bf16: 47 rows each 94 (82) / 75 (83), 48 rows the
//    same, 96 rows 109 (104) / 82 (115), 128 rows 112 (115) / 86 (123).  fp32 products, which take
//    16 times as long, want two tiles for each: 2000 rows, 2 experts, 512 x 2048 (272
//    tiles): 43 (69).
// What the mean costs where few experts hold all rows, 2048 x 1408, bf16: 4 of 64, 16384
// rows, nothing; 4 of 128, 16384 rows, 112 (256 x 256: 102) / 119 (99); 4 of 128, 4096 rows, 63
// (128 x 128: 37) / 71 (40); 1 of 64, 2048 rows, 33 (256 x 256: 23) / 34 (23).
template <typename T, int KIND, typename TO, int LOAD>
int launch_loaded(int pk, const XArgs& a, hipStream_t stream) {
  const int64_t cus = device_cus();
  const int64_t avg = a.n / a.experts;
  auto tiles = [&](int t) {
    if (KIND == X_DW) return cdiv(a.m, t) * cdiv(a.k, t) * a.experts;
    return (cdiv(a.n, t) + a.experts / 2) * cdiv(KIND == X_FWD ? a.m : a.k, t);
  };
  constexpr int KB = 128 / sizeof(T);   // l per slab
  constexpr bool dw = KIND == X_DW;
  const int64_t sum = dw ? avg : KIND == X_FWD ? a.k : a.m;
  if (dw ? tiles(64) <= cus && sum >= 8 * KB : (avg <= 32 || tiles(64) <= 2 * cus) && sum >= 4 * KB)
    return launch_split<T, KIND, TO, LOAD>(pk, a, stream);
  if constexpr (dw && LOAD == X_DIRECT) {
    if (sum <= 2 * KB && tiles(128) >= cus) return launch_tile<T, KIND, TO, 128, 128, 2, 2, 1, LOAD>(pk, a, stream);
  }
  if constexpr (sizeof(T) == 2) {
    if ((dw || avg >= 160) && tiles(256) >= cus)
      return launch_tile<T, KIND, TO, 256, 256, 2, 4, 2, LOAD>(pk, a, stream);
  }
  if ((dw || avg >= 48) && tiles(128) >= (sizeof(T) == 2 ? cus : 2 * cus))
    return launch_tile<T, KIND, TO, 128, 128, 2, 2, 2, LOAD>(pk, a, stream);
  return launch_tile<T, KIND, TO, 64, 64, 2, 2, LOAD == X_DIRECT ? 3 : 2, LOAD>(pk, a, stream);
}

template <typename T, int KIND, typename TO>
int launch_typed(int pk, const XCall& c, hipStream_t stream) {
  constexpr int EPC = 16 / sizeof(T);
  // widths of the operands' rows: k and m, k alone for X_FWD
  if (c.a.k < EPC || (KIND != X_FWD && c.a.m < EPC))
    return launch_tile<T, KIND, TO, 64, 64, 2, 2, 2, X_SINGLE>(pk, c.a, stream);
  if (c.p_direct && c.q_direct) return launch_loaded<T, KIND, TO, X_DIRECT>(pk, c.a, stream);
  // X_FWD's operands share the row width, so there one alone is rare
  if constexpr (KIND != X_FWD) {
    if (c.p_direct) return launch_loaded<T, KIND, TO, X_P_DIRECT>(pk, c.a, stream);
    if (c.q_direct) return launch_loaded<T, KIND, TO, X_Q_DIRECT>(pk, c.a, stream);
  }
  return launch_loaded<T, KIND, TO, X_PIECE>(pk, c.a, stream);
}

template <int KIND>
int launch_expert(int pk, const XCall& c, hipStream_t stream) {
  if (c.dtype == MO_F32) return launch_typed<float, KIND, float>(pk, c, stream);
  if (c.out == MO_F32) return launch_typed<bf16_t, KIND, float>(pk, c, stream);
  return launch_typed<bf16_t, KIND, bf16_t>(pk, c, stream);
}

}  // namespace mo
