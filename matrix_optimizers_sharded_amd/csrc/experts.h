// Products grouped by expert over ragged row segments, on the matrix cores.
//
// Rows of x (n x k) and dy (n x m) are in the order of their expert; expert e holds
// rows o[e] .. o[e+1]-1 and a weight w[e] (m x k).  Three products:
//   X_FWD  y[r][j]    = sum_k x[r][k] w[e][j][k]        rows of the segment x m
//   X_DX   dx[r][j]   = sum_m dy[r][m] w[e][m][j]       rows of the segment x k
//   X_DW   dw[e][i][j] = sum_r dy[r][i] x[r][j]         m x k, the sum over the segment
// Each is C[i][j] = sum_l P(i, l) Q(l, j).  An operand whose sum index l runs along its
// rows in memory ("K-major") is staged as rows of 128 bytes of l; one whose rows ARE
// the sum index ("N-major": w in X_DX, both in X_DW) as [column block][l][128 bytes],
// read through gfx950's transposing LDS reads, so no operand is ever transposed in
// memory.  Sums are fp32 in the matrix cores' accumulators; each result is rounded
// once, to the output type.
//
// Segments come from the device, so the tile list does too: every block sums the
// segments' tiles in LDS and finds its own.  Offsets are clamped to [0, n] and made
// ascending, so that a bad table can give wrong rows but no access out of range and no row
// that nobody or more than one writes.  Rows that no segment
// holds (before o[0], from o[E] on) get zeros: they are tiles with an empty sum.  An
// expert without rows gets a zero weight gradient the same way.
//
// What bounds them.  Many rows an expert: the matrix cores, whose clock drops under this
// load.  16384 rows over 8 experts, 4096 x 11008, bf16: 1290 / 1300 / 1290 us for X_FWD /
// X_DX / X_DW, 1.14 PFLOP/s; one expert and whole rounds of tiles, 8192^3: 1.25-1.28.  The
// rest goes to ragged ends, the last round of tiles and each tile's own start and end (a
// compute unit holds one 256 x 256 tile, so its stores overlap no product).  Few rows: the
// weights' way from HBM, 48 rows over 8 experts, 2048 x 5632: 35 us, 5.3 TB/s (29 with weights
// that the caches still hold in part).  Short sums: the
// weight gradients' stores.  Between them, 128 rows an expert, 2048 x 1400: 3.7 TB/s
// (X_FWD), 5.6 (X_DW).
#pragma once

#include "gemm.h"

namespace mo {

enum XKind { X_FWD = 0, X_DX = 1, X_DW = 2 };

// How operands reach LDS: straight, where all rows start 16-byte aligned and end on 16
// bytes (one operand or both); through registers in pieces of 16 bytes; or element by
// element, for rows shorter than that.
enum XLoad { X_PIECE = 0, X_P_DIRECT = 1, X_Q_DIRECT = 2, X_DIRECT = 3, X_SINGLE = 4 };

constexpr int X_MAX_EXPERTS = 1024;

struct XArgs {
  const void* P;
  const void* Q;
  void* C;
  const int32_t* offsets;   // experts + 1
  int64_t ldp, ldq, ldc;    // row pitches in elements
  int64_t n;                // rows of x, dy
  int32_t experts, k, m;
  int32_t vec_out;          // results can be stored 16 bytes at a time (aligned rows)
  int32_t slots;            // blocks that the device runs at a time
  int64_t first_block;      // of this launch
};

// N 16-byte-per-lane loads straight into LDS (see load_lds16x4).
__device__ inline void load_lds16x2(i32x4_t rsrc, const uint32_t (&lds)[2], const uint32_t (&voff)[2]) {
  i32x4_t r;
#pragma unroll
  for (int c = 0; c < 4; ++c) r[c] = __builtin_amdgcn_readfirstlane(rsrc[c]);
  const uint32_t l0 = __builtin_amdgcn_readfirstlane(lds[0]), l1 = __builtin_amdgcn_readfirstlane(lds[1]);
  uint32_t saved;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %1\n\ts_nop 0\n\tbuffer_load_dwordx4 %3, %5, 0 offen lds\n\t"
      "s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %4, %5, 0 offen lds\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(saved)
      : "s"(l0), "s"(l1), "v"(voff[0]), "v"(voff[1]), "s"(r)
      : "memory");
}

// 16 bytes from an address aligned to the element only; and to one.
struct __attribute__((packed, aligned(2))) Bytes16 { u32x4_t v; };
struct __attribute__((packed, aligned(4))) Bytes16x4 { u32x4_t v; };
template <typename T> struct Loose { typedef Bytes16x4 type; };
template <> struct Loose<bf16_t> { typedef Bytes16 type; };
template <typename T>
__device__ inline void store16_loose(T* p, u32x4_t v) {
  reinterpret_cast<gptr<typename Loose<T>::type>>(global(p))->v = v;
}

// Which tile a block computes.
struct XTile {
  int64_t row0;    // X_FWD, X_DX: first row of C (and P)
  int rows;        // rows of this segment from there on (X_DW: rows of C from i0 on)
  int e;           // expert, or -1: rows of no segment
  int i0, j0;      // X_DW: first row of C; first column of C
  int64_t l0;      // X_DW: first row of the segment
  int L;           // length of the sum
};

// Segment tables in LDS: seg[s] is the first item of segment s, s < experts + 2 (the
// rows before o[0], the experts, the rows from o[experts] on).
struct XSegs {
  int32_t lo[X_MAX_EXPERTS + 2];
  int32_t hi[X_MAX_EXPERTS + 2];
  int32_t begin[X_MAX_EXPERTS + 3];
};

__device__ inline int clamp_row(int v, int64_t n) {
  return v < 0 ? 0 : v > n ? static_cast<int>(n) : v;
}

// Items (tiles) of X_FWD and X_DX: every segment's row tiles times `ct` column tiles,
// as a running sum.  One wave, 64 segments at a time.  A bound below an earlier one is
// raised to it, so segments share no row and cover [0, n) whatever the table holds: every
// row is written once, and the grid's bound (row_tiles) and 32-bit sums hold.
template <int TM>
__device__ inline void x_segments(const XArgs& a, int ct, XSegs& s) {
  const int lane = threadIdx.x & 63;
  const int S = a.experts + 2;
  if (threadIdx.x < 64) {
    int run = 0, top = 0;   // top: the end of the segments so far
    for (int s0 = 0; s0 < S; s0 += 64) {
      const int i = s0 + lane;
      int lo = 0, hi = 0;
      if (i < S) {
        lo = i == 0 ? 0 : clamp_row(a.offsets[i - 1], a.n);
        hi = i == S - 1 ? static_cast<int>(a.n) : clamp_row(a.offsets[i], a.n);
      }
      if (__ballot(i < S && (hi < lo || lo < top)) != 0) {   // not for an ascending table
        hi = max(hi, top);
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
          const int up = __shfl_up(hi, d);
          if (lane >= d) hi = max(hi, up);
        }
        lo = __shfl_up(hi, 1);
        if (lane == 0) lo = top;
      }
      top = __shfl(hi, 63);
      if (i < S) {
        s.lo[i] = lo;
        s.hi[i] = hi;
      }
      int v = (hi - lo + TM - 1) / TM * ct;
      int inc = v;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int up = __shfl_up(inc, d);
        if (lane >= d) inc += up;
      }
      if (i < S) s.begin[i] = run + inc - v;
      run += __shfl(inc, 63);
    }
    if (lane == 0) s.begin[S] = run;
  }
  __syncthreads();
}

template <typename T, int KIND, int TM_, int TN_, int WR_, int WC_, int STAGES, typename TO, int LOAD>
struct XGemm {
  static constexpr int TM = TM_, TN = TN_, WR = WR_, WC = WC_;
  static constexpr int NW = WR * WC, NT = 64 * NW;
  static constexpr int WM = TM / WR, WN = TN / WC;       // a wave's part of the tile
  static constexpr int NA = WM / 32, NBX = WN / 32;       // its 32 x 32 blocks
  static constexpr int ES = sizeof(T);
  static constexpr int KB = 128 / ES;                     // l per slab
  static constexpr int EPC = 16 / ES;                     // elements per 16-byte chunk
  static constexpr bool PN = KIND == X_DW, QN = KIND != X_FWD;   // N-major operands
  static constexpr bool PD = LOAD & X_P_DIRECT, QD = LOAD & X_Q_DIRECT;
  static constexpr int P_BYTES = TM * 128, Q_BYTES = TN * 128, STAGE = P_BYTES + Q_BYTES;
  // a wave's staging area for results: 32 rows of its columns, rows 16 bytes apart in
  // banks
  static constexpr int OUT_PITCH = WN * static_cast<int>(sizeof(TO)) + 16;
  static constexpr int OUT_BYTES = 32 * OUT_PITCH;
  static constexpr int LDS_BYTES = STAGES * STAGE > NW * OUT_BYTES ? STAGES * STAGE : NW * OUT_BYTES;
  static constexpr int RG = KB / 8;                       // 8-row groups of an N-major block
  // with bf16 operands and 8 waves one wave per SIMD issues the loads of two (see gemm.h)
  static constexpr int LOADERS = (NW == 8 && ES == 2) ? 4 : NW;
  static constexpr int UP = TM / 8 / NW, UQ = TN / 8 / NW;        // 1 KiB units per wave and slab
  static constexpr int UPL = TM / 8 / LOADERS, UQL = TN / 8 / LOADERS;
  static_assert(TM % (8 * NW) == 0 && TN % (8 * NW) == 0, "whole units per wave");
  static_assert((!PN || TM % KB == 0) && (!QN || TN % KB == 0), "whole N-major column blocks");
  // Smaller tiles of the same waves (see k_expert): half of the rows, and half of the
  // rows and columns, with deeper rings in about the same LDS.
  static constexpr bool SPLITS = WM >= 64 && WN >= 64;
  typedef XGemm<T, KIND, TM / 2, TN, WR, WC, STAGES == 1 ? 1 : LOAD == X_DIRECT ? 3 : 2, TO, LOAD> Half;
  typedef XGemm<T, KIND, TM / 2, TN / 2, WR, WC, (LOAD == X_DIRECT && STAGES > 1) ? 4 : 2, TO, LOAD> Quarter;

  // One operand of a tile: its first byte, its pitch, and how far it reaches.
  struct Operand {
    const unsigned char* base;
    int64_t pitch;   // bytes
    int64_t bytes;   // bytes from base that may be read
    int rows;        // K-major: rows that exist; N-major: columns that exist
  };

  // byte offset of unit u, this lane, slab-relative; K-major rows advance along the
  // tile, N-major rows along l
  template <bool NM>
  static __device__ inline uint32_t lane_off(int u, int lane, int64_t pitch, int& row, int& chunk) {
    if constexpr (!NM) {
      row = 8 * u + (lane >> 3);
      chunk = (lane & 7) ^ swz(row);
      return static_cast<uint32_t>(row * pitch) + chunk * 16;
    } else {
      row = (u % RG) * 8 + (lane >> 3);
      chunk = (u / RG) * 8 + ((lane & 7) ^ swz_tr(row));
      return static_cast<uint32_t>(row * pitch) + chunk * 16;
    }
  }

  // ---- DMA: slab kt of an operand straight into LDS.  Rows past the end and, in the
  // last slab of a K-major operand, chunks past L lie outside the buffer resource and
  // arrive as zeros.
  template <bool NM, int U>
  static __device__ inline void dma(const Operand& o, int kt, int L, uint32_t lds, int wave, int lane) {
    if (wave >= LOADERS) return;
    const int64_t skip = NM ? static_cast<int64_t>(kt) * KB * o.pitch : static_cast<int64_t>(kt) * 128;
    int64_t left = o.bytes - skip;
    left = left < 0 ? 0 : left > 0x7fffff00 ? 0x7fffff00 : left;
    const i32x4_t r = buffer_rsrc(o.base + skip, static_cast<uint32_t>(left));
    const bool tail = !NM && (kt + 1) * KB > L;
    uint32_t l[U], v[U];
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const int u = q * LOADERS + wave;
      int row, chunk;
      v[q] = lane_off<NM>(u, lane, o.pitch, row, chunk);
      if (tail && kt * KB + chunk * EPC >= L) v[q] = 0x80000000u;
      l[q] = lds + u * 1024;
    }
    if constexpr (U % 4 == 0) {
#pragma unroll
      for (int q = 0; q < U; q += 4) {
        const uint32_t l4[4] = {l[q], l[q + 1], l[q + 2], l[q + 3]}, v4[4] = {v[q], v[q + 1], v[q + 2], v[q + 3]};
        load_lds16x4(r, l4, v4, 0);
      }
    } else {
#pragma unroll
      for (int q = 0; q < U; q += 2) {
        const uint32_t l2[2] = {l[q], l[q + 1]}, v2[2] = {v[q], v[q + 1]};
        load_lds16x2(r, l2, v2);
      }
    }
  }

  // ---- through registers: rows that start at any element.  Away from the edges a piece
  // of 16 bytes is one load.  At the edges the 16 bytes move back to where the row still
  // has them, and put() shifts the elements into place and clears what lies past the end:
  // every load is made by all lanes at once, none waits for another.  (Pieces at the
  // edges loaded element by element: 58 us instead of 29 for 760 rows over 4 experts,
  // 839 x 1739.  Loads of whole dwords, five for a piece at an odd bf16 element, instead
  // of four dwords 2 bytes off: 750 us instead of 500 for 4095 x 5631.)
  //
  // Where a piece and its load begin, in bytes from the slab's first; its elements that
  // exist.
  struct Spot {
    int at, window, have;
  };
  template <bool NM>
  static __device__ inline Spot spot(const Operand& o, int kt, int L, int u, int lane) {
    int row, chunk;
    (void)lane_off<NM>(u, lane, 0, row, chunk);
    const int left = NM ? L - kt * KB : o.rows;                  // rows of the slab, > 0
    const int c = (NM ? 0 : kt * KB) + chunk * EPC, cols = NM ? o.rows : L;
    const int start = min(row, left - 1) * static_cast<int>(o.pitch);
    Spot s;
    s.at = start + c * ES;
    s.window = min(s.at, start + cols * ES - 16);
    s.have = NM && row >= left ? 0 : min(max(cols - c, 0), EPC);
    return s;
  }
  // Away from the edges every piece is whole.  (Rows past the end of a K-major operand
  // repeat its last: they only reach results that are not stored.)
  template <bool NM, int U>
  static __device__ inline bool inside(const Operand& o, int kt, int L) {
    return (kt + 1) * KB <= L && (!NM || o.rows >= U * 8 * NW);
  }
  template <bool NM, int U>
  static __device__ inline void fetch(const Operand& o, int kt, int L, int wave, int lane, u32x4_t (&buf)[U]) {
    const unsigned char* slab = o.base + (NM ? static_cast<int64_t>(kt) * KB * o.pitch : 0);
    typedef __attribute__((address_space(1))) const unsigned char* bytes_t;
    const bytes_t p = (bytes_t)slab;
    typedef gptr<const typename Loose<T>::type> piece_t;
    if constexpr (LOAD == X_SINGLE) {
#pragma unroll
      for (int q = 0; q < U; ++q) {
        const Spot s = spot<NM>(o, kt, L, q * NW + wave, lane);
        typedef typename std::conditional<ES == 2, uint16_t, uint32_t>::type word_t;
        const auto g = global(reinterpret_cast<const word_t*>(slab + s.at));
        uint32_t w[EPC];
#pragma unroll
        for (int i = 0; i < EPC; ++i) w[i] = i < s.have ? g[i] : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) buf[q][i] = ES == 2 ? w[i * EPC / 4] | (w[i * EPC / 4 + EPC / 4 - 1] << 16) : w[i];
      }
    } else if (inside<NM, U>(o, kt, L)) {
#pragma unroll
      for (int q = 0; q < U; ++q) {
        int row, chunk;
        (void)lane_off<NM>(q * NW + wave, lane, 0, row, chunk);
        if constexpr (!NM) row = min(row, o.rows - 1);
        const uint32_t at = static_cast<uint32_t>(row * static_cast<int>(o.pitch)) + chunk * 16;
        buf[q] = reinterpret_cast<piece_t>(p + (NM ? 0 : kt * 128) + at)->v;
      }
    } else {
#pragma unroll
      for (int q = 0; q < U; ++q)
        buf[q] = reinterpret_cast<piece_t>(p + spot<NM>(o, kt, L, q * NW + wave, lane).window)->v;
    }
  }
  template <bool NM, int U>
  static __device__ inline void put(const Operand& o, int kt, int L, u32x4_t (&buf)[U], unsigned char* lds, int wave,
                                    int lane) {
    if (LOAD != X_SINGLE && !inside<NM, U>(o, kt, L)) {
#pragma unroll
      for (int q = 0; q < U; ++q) {
        const Spot s = spot<NM>(o, kt, L, q * NW + wave, lane);
        const int by = s.at - s.window;
        const bool two = by & 8, one = by & 4;
        uint32_t v0 = buf[q][0], v1 = buf[q][1], v2 = buf[q][2], v3 = buf[q][3];
        v0 = two ? v2 : v0;
        v1 = two ? v3 : v1;
        v0 = one ? v1 : v0;
        v1 = one ? v2 : v1;
        v2 = one ? v3 : v2;
        if constexpr (ES == 2) {
          v0 = __builtin_amdgcn_alignbyte(v1, v0, by & 2);
          v1 = __builtin_amdgcn_alignbyte(v2, v1, by & 2);
          v2 = __builtin_amdgcn_alignbyte(v3, v2, by & 2);
          v3 = __builtin_amdgcn_alignbyte(0u, v3, by & 2);
        }
        u32x4_t v = {v0, v1, v2, v3};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int n = s.have - i * EPC / 4;
          v[i] = n <= 0 ? 0 : (ES == 2 && n == 1) ? v[i] & 0xffffu : v[i];
        }
        buf[q] = v;
      }
    }
#pragma unroll
    for (int q = 0; q < U; ++q)
      *reinterpret_cast<u32x4_t*>(lds + (q * NW + wave) * 1024 + lane * 16) = buf[q];
  }

  // at most min(left, MOST) slabs' loads still in flight (none for left < 1)
  template <int MOST>
  static __device__ inline void wait_slabs(int left) {
    static_assert(MOST * (UPL + UQL) < 64, "vmcnt is a 6-bit field");
    if constexpr (MOST > 0) {
      if (left >= MOST)
        __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0(MOST * (UPL + UQL)));
      else
        wait_slabs<MOST - 1>(left);
    } else {
      __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0(0));
    }
  }

  typedef typename Mfma<T>::frag frag_t;

  // the operand fragment of 32 rows (columns) from r0 on, k16 (bf16) or 8 l (fp32) step kk
  template <bool NM>
  static __device__ inline frag_t frag(const unsigned char* s, int r0, int kk, int lane) {
    const int l32 = lane & 31, half = lane >> 5, c = 2 * kk + half;
    if constexpr (!NM) {
      const int r = r0 + l32;
      return *reinterpret_cast<const frag_t*>(s + r * 128 + ((c ^ swz(r)) << 4));
    } else if constexpr (ES == 2) {
      const int trow = 8 * half + ((lane & 15) >> 2), tcol = 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
      const int n = r0 + tcol, nb = (n % KB) * 2, k = 16 * kk + trow;
      const unsigned char* q = s + (n / KB) * (KB * 128) + k * 128 + ((((nb >> 4) ^ swz_tr(k)) << 4) | (nb & 15));
      const bf16x4_t lo = lds_read_tr16(q), hi = lds_read_tr16(q + 4 * 128);
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
      const int n = r0 + l32, nb = (n % KB) * 4;
      const unsigned char* col = s + (n / KB) * (KB * 128);
      frag_t f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int k = 4 * c + e;
        f[e] = *reinterpret_cast<const float*>(col + k * 128 + ((((nb >> 4) ^ swz_tr(k)) << 4) | (nb & 15)));
      }
      return f;
    }
  }

  static constexpr int KST = CHUNKS / 2;   // MFMA steps per slab

  static __device__ inline void read_frags(const unsigned char* st, int kk, int wm, int wn, int lane,
                                           frag_t (&A)[NA], frag_t (&B)[NBX]) {
#pragma unroll
    for (int x = 0; x < NA; ++x) A[x] = frag<PN>(st, wm + 32 * x, kk, lane);
#pragma unroll
    for (int x = 0; x < NBX; ++x) B[x] = frag<QN>(st + P_BYTES, wn + 32 * x, kk, lane);
  }
  static __device__ inline void mma(f32x16_t (&acc)[NA][NBX], const frag_t (&A)[NA], const frag_t (&B)[NBX]) {
#pragma unroll
    for (int x = 0; x < NA; ++x)
#pragma unroll
      for (int y = 0; y < NBX; ++y) Mfma<T>::mma(acc[x][y], A[x], B[y]);
  }
  // LDS reads and MFMAs of a step side by side (see gemm.h)
  static __device__ inline void interleave() {
    constexpr int RA = PN ? (ES == 2 ? 2 : 4) : 1, RB = QN ? (ES == 2 ? 2 : 4) : 1;
    constexpr int NR = NA * RA + NBX * RB, NM = NA * NBX * (ES == 2 ? 1 : 4);
    constexpr int NP = NR < NM ? NR : NM;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    }
    if constexpr (NM > NP) __builtin_amdgcn_sched_group_barrier(0x008, NM - NP, 0);
    if constexpr (NR > NP) __builtin_amdgcn_sched_group_barrier(0x100, NR - NP, 0);
    __builtin_amdgcn_sched_barrier(0);
  }

  // a tile's two operands
  static __device__ inline void operands(const XArgs& a, const XTile& t, Operand& P, Operand& Q) {
    const int L = t.L;
    P.pitch = a.ldp * ES;
    Q.pitch = a.ldq * ES;
    const unsigned char* p0 = static_cast<const unsigned char*>(a.P);
    const unsigned char* q0 = static_cast<const unsigned char*>(a.Q);
    if constexpr (KIND == X_DW) {
      P.base = p0 + t.l0 * P.pitch + static_cast<int64_t>(t.i0) * ES;
      Q.base = q0 + t.l0 * Q.pitch + static_cast<int64_t>(t.j0) * ES;
      P.rows = a.m - t.i0;
      Q.rows = a.k - t.j0;
      P.bytes = static_cast<int64_t>(L - 1) * P.pitch + static_cast<int64_t>(P.rows) * ES;
      Q.bytes = static_cast<int64_t>(L - 1) * Q.pitch + static_cast<int64_t>(Q.rows) * ES;
    } else {
      const int64_t we = static_cast<int64_t>(t.e < 0 ? 0 : t.e) * a.m * Q.pitch;
      P.base = p0 + t.row0 * P.pitch;
      P.rows = t.rows;
      P.bytes = static_cast<int64_t>(t.rows - 1) * P.pitch + static_cast<int64_t>(L) * ES;
      if constexpr (KIND == X_FWD) {
        Q.base = q0 + we + static_cast<int64_t>(t.j0) * Q.pitch;
        Q.rows = a.m - t.j0;
        Q.bytes = static_cast<int64_t>(Q.rows - 1) * Q.pitch + static_cast<int64_t>(L) * ES;
      } else {
        Q.base = q0 + we + static_cast<int64_t>(t.j0) * ES;
        Q.rows = a.k - t.j0;
        Q.bytes = static_cast<int64_t>(L - 1) * Q.pitch + static_cast<int64_t>(Q.rows) * ES;
      }
    }
  }

  static __device__ inline void run(const XArgs& a, unsigned char* smem, const XTile& t) {
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = (wave / WC) * WM, wn = (wave % WC) * WN;
    const int ncols = KIND == X_FWD ? a.m : a.k;
    f32x16_t acc[NA][NBX];
#pragma unroll
    for (int x = 0; x < NA; ++x)
#pragma unroll
      for (int y = 0; y < NBX; ++y)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[x][y][r] = 0.f;

    const int L = t.L, nk = (L + KB - 1) / KB;
    Operand P, Q;
    operands(a, t, P, Q);

    frag_t fa[2][NA], fb[2][NBX];
    if (nk > 0) {
      if constexpr (LOAD == X_DIRECT) {
        const uint32_t base = lds_addr(smem);
        auto issue = [&](int kt, int stage) {
          dma<PN, UPL>(P, kt, L, base + stage * STAGE, wave, lane);
          dma<QN, UQL>(Q, kt, L, base + stage * STAGE + P_BYTES, wave, lane);
        };
        if constexpr (STAGES == 1) {
          // one slab at a time: the other blocks of the compute unit hide its latency
          for (int kt = 0; kt < nk; ++kt) {
            issue(kt, 0);
            wait_slabs<0>(0);
            __syncthreads();
            read_frags(smem, 0, wm, wn, lane, fa[0], fb[0]);
#pragma unroll
            for (int kk = 0; kk < KST; ++kk) {
              if (kk + 1 < KST) read_frags(smem, kk + 1, wm, wn, lane, fa[(kk + 1) & 1], fb[(kk + 1) & 1]);
              mma(acc, fa[kk & 1], fb[kk & 1]);
            }
            __syncthreads();
          }
        } else {
#pragma unroll
          for (int s = 0; s < STAGES; ++s)
            if (s < nk) issue(s, s);
          wait_slabs<STAGES - 1>(nk - 1);
          __syncthreads();
          read_frags(smem, 0, wm, wn, lane, fa[0], fb[0]);
          int stage = 0;
          for (int kt = 0; kt < nk; ++kt) {
            const unsigned char* st = smem + stage * STAGE;
#pragma unroll
            for (int kk = 0; kk < KST - 1; ++kk) {
              read_frags(st, kk + 1, wm, wn, lane, fa[(kk + 1) & 1], fb[(kk + 1) & 1]);
              mma(acc, fa[kk & 1], fb[kk & 1]);
              interleave();
            }
            // slab kt + 1 is in for everyone, and nobody reads slab kt any more; on the
            // last slab the reads below fetch unused fragments
            const int next = stage + 1 == STAGES ? 0 : stage + 1;
            wait_slabs<(STAGES > 2 ? STAGES - 2 : 0)>(nk - kt - 2);
            __syncthreads();
            read_frags(smem + next * STAGE, 0, wm, wn, lane, fa[0], fb[0]);
            mma(acc, fa[(KST - 1) & 1], fb[(KST - 1) & 1]);
            interleave();
            if (kt + STAGES < nk) issue(kt + STAGES, stage);
            stage = next;
          }
        }
      } else {
        u32x4_t bp[UP], bq[UQ];
        const uint32_t base = lds_addr(smem);
        // slab kt on its way: to the registers, or into a stage that nobody reads any more
        auto start = [&](int kt, int stage) {
          if constexpr (PD) dma<PN, UPL>(P, kt, L, base + stage * STAGE, wave, lane);
          else fetch<PN, UP>(P, kt, L, wave, lane, bp);
          if constexpr (QD) dma<QN, UQL>(Q, kt, L, base + stage * STAGE + P_BYTES, wave, lane);
          else fetch<QN, UQ>(Q, kt, L, wave, lane, bq);
        };
        auto finish = [&](int kt, int stage) {
          if constexpr (!PD) put<PN, UP>(P, kt, L, bp, smem + stage * STAGE, wave, lane);
          if constexpr (!QD) put<QN, UQ>(Q, kt, L, bq, smem + stage * STAGE + P_BYTES, wave, lane);
          if constexpr (PD || QD) wait_slabs<0>(0);
          __syncthreads();
        };
        start(0, 0);
        finish(0, 0);
        for (int kt = 0; kt < nk; ++kt) {
          const unsigned char* st = smem + (kt & 1) * STAGE;
          if (kt + 1 < nk) start(kt + 1, (kt + 1) & 1);
          read_frags(st, 0, wm, wn, lane, fa[0], fb[0]);
#pragma unroll
          for (int kk = 0; kk < KST; ++kk) {
            if (kk + 1 < KST) read_frags(st, kk + 1, wm, wn, lane, fa[(kk + 1) & 1], fb[(kk + 1) & 1]);
            mma(acc, fa[kk & 1], fb[kk & 1]);
          }
          if (kt + 1 < nk) finish(kt + 1, (kt + 1) & 1);
        }
      }
    }
    __syncthreads();   // the ring becomes the staging area

    // Results leave as 16-byte pieces of rows.  Lane l, register r of a 32 x 32 block
    // hold row 8*(r/4) + 4*(l/32) + r%4, column l%32.
    constexpr int EPV = 16 / sizeof(TO);       // elements per piece
    constexpr int PPR = WN / EPV;              // pieces per row
    unsigned char* stg = smem + wave * OUT_BYTES;
    const int half = lane >> 5, l32 = lane & 31;
    TO* C = static_cast<TO*>(a.C) +
            (KIND == X_DW ? static_cast<int64_t>(t.e) * a.m * a.ldc + static_cast<int64_t>(t.i0) * a.ldc
                          : t.row0 * a.ldc);
#pragma unroll
    for (int x = 0; x < NA; ++x) {
#pragma unroll
      for (int y = 0; y < NBX; ++y)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int row = 8 * (r >> 2) + 4 * half + (r & 3);
          *reinterpret_cast<TO*>(stg + row * OUT_PITCH + (32 * y + l32) * sizeof(TO)) = from_f32<TO>(acc[x][y][r]);
        }
      // the wave's own LDS accesses execute in order
#pragma unroll
      for (int q = 0; q < 32 * PPR / 64; ++q) {
        const int at = q * 64 + lane, row = at / PPR, piece = at % PPR;
        const int i = wm + 32 * x + row, j = t.j0 + wn + piece * EPV;
        if (i < t.rows && j < ncols) {
          const u32x4_t v = *reinterpret_cast<const u32x4_t*>(stg + row * OUT_PITCH + piece * 16);
          TO* c = C + static_cast<int64_t>(i) * a.ldc + j;
          if (j + EPV <= ncols) {
            // past the caches, where the operands of other tiles are: 16 to 27% less
            // time for weight gradients of short sums, 3% for products of long ones
            if (a.vec_out)
              __builtin_nontemporal_store(v, reinterpret_cast<gptr<u32x4_t>>(global(c)));
            else
              store16_loose(c, v);
          } else {
            TO x8[EPV];
            __builtin_memcpy(x8, &v, 16);
#pragma unroll
            for (int e = 0; e < EPV; ++e)
              if (j + e < ncols) global(c)[e] = x8[e];
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
};

// LDS of a kernel: the largest that one of its tiles takes
template <typename G, bool SPLITS = G::SPLITS>
struct XLds {
  static constexpr int bytes = G::LDS_BYTES;
};
template <typename G>
struct XLds<G, true> {
  static constexpr int h = G::Half::LDS_BYTES, q = G::Quarter::LDS_BYTES, b = h > q ? h : q;
  static constexpr int bytes = G::LDS_BYTES > b ? G::LDS_BYTES : b;
};

// Which item block b takes, and which part of it.  The device runs `slots` blocks at a
// time, so the last total % slots items would leave most of it idle for a whole tile's
// time.  Where they are few they are cut, each into quarters or into halves of its rows.
struct XPart {
  int64_t item;   // < 0: none
  int ways, sub;  // 1, 2 or 4 parts; this block's
};
template <bool SPLITS>
__device__ inline XPart x_part(int64_t b, int64_t total, int slots) {
  const int64_t rest = SPLITS ? total % slots : 0;
  const int ways = 4 * rest <= slots ? 4 : 2 * rest <= slots ? 2 : 1;
  const int64_t whole = ways > 1 ? total - rest : total;
  if (b < whole) return {xcd_remap(b, whole), 1, 0};
  const int64_t at = b - whole;
  if (ways == 1 || at >= rest * ways) return {-1, 1, 0};
  return {whole + at / ways, ways, static_cast<int>(at % ways)};
}

// The tile of this block, or false if it has none: an item of the list, found through
// the segment table (LDS, freed on return), and where the list's end is cut a part of it.
template <int KIND, int TM, int TN, bool SPLITS>
__device__ inline bool x_tile(const XArgs& a, unsigned char* smem, XTile& t, int& ways) {
  const int ncols = KIND == X_FWD ? a.m : a.k;
  const int ct = (ncols + TN - 1) / TN;
  XPart part;
  if constexpr (KIND == X_DW) {
    const int ti = (a.m + TM - 1) / TM;
    const int64_t per = static_cast<int64_t>(ti) * ct, total = per * a.experts;
    part = x_part<SPLITS>(a.first_block + blockIdx.x, total, a.slots);
    if (part.item < 0) return false;
    t.e = static_cast<int>(part.item / per);
    int i, j;
    rect_tile(part.item - t.e * per, ti, ct, i, j);
    t.i0 = i * TM;
    t.j0 = j * TN;
    t.rows = a.m - t.i0;
    t.row0 = 0;
    const int lo = clamp_row(a.offsets[t.e], a.n), hi = clamp_row(a.offsets[t.e + 1], a.n);
    t.l0 = lo;
    t.L = hi > lo ? hi - lo : 0;
  } else {
    XSegs& s = *reinterpret_cast<XSegs*>(smem);
    x_segments<TM>(a, ct, s);
    const int S = a.experts + 2, total = s.begin[S];
    part = x_part<SPLITS>(a.first_block + blockIdx.x, total, a.slots);
    if (part.item < 0) return false;
    const int item = static_cast<int>(part.item);
    int lo = 0, hi = S - 1;   // the last segment that begins at or before the item
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s.begin[mid] <= item) lo = mid; else hi = mid - 1;
    }
    const int size = s.hi[lo] - s.lo[lo], rt = (size + TM - 1) / TM;
    int i, j;
    rect_tile(item - s.begin[lo], rt, ct, i, j);
    t.row0 = s.lo[lo] + static_cast<int64_t>(i) * TM;
    t.rows = size - i * TM;
    t.e = (lo == 0 || lo == S - 1) ? -1 : lo - 1;
    t.i0 = 0;
    t.j0 = j * TN;
    t.l0 = 0;
    t.L = t.e < 0 ? 0 : (KIND == X_FWD ? a.k : a.m);
    __syncthreads();   // the table's memory becomes the ring
  }
  ways = part.ways;
  if constexpr (SPLITS) {
    if (ways > 1) {
      const int down = (ways == 4 ? part.sub >> 1 : part.sub) * (TM / 2);
      const int across = (ways == 4 ? part.sub & 1 : 0) * (TN / 2);
      t.rows -= down;
      t.j0 += across;
      if (KIND == X_DW) t.i0 += down; else t.row0 += down;
      if (t.rows <= 0 || t.j0 >= ncols) return false;
    }
  }
  t.e = __builtin_amdgcn_readfirstlane(t.e);
  t.L = __builtin_amdgcn_readfirstlane(t.L);
  t.rows = __builtin_amdgcn_readfirstlane(t.rows);
  return true;
}

// One block per tile, or per part of a tile at the end of the list.  The grid is an
// upper bound of both (x_blocks): for X_FWD and X_DX the segments' sizes are not known
// on the host.  A tile whose rows end in its first half takes the half tile.
template <typename G, int KIND>
__global__ __launch_bounds__(G::NT) void k_expert(XArgs a) {
  __shared__ __attribute__((aligned(1024))) unsigned char smem[XLds<G>::bytes];
  static_assert(KIND == X_DW || sizeof(XSegs) <= sizeof(smem), "segment table");
  XTile t;
  int ways;
  if (!x_tile<KIND, G::TM, G::TN, G::SPLITS>(a, smem, t, ways)) return;
  if constexpr (G::SPLITS) {
    if (ways == 4) {
      G::Quarter::run(a, smem, t);
      return;
    }
    if (ways == 2 || t.rows <= G::TM / 2) {
      G::Half::run(a, smem, t);
      return;
    }
  }
  G::run(a, smem, t);
}

// Few tiles and a long sum: KW waves share a tile of 32 rows (64 where an N-major slab
// is that wide) and 64 columns, each with its own part of the sum (slabs w, w + KW, ...)
// and its own slab in LDS, so no wave waits for another before the end, where the KW
// partial tiles are added in the waves' order.
template <typename T, int KIND, typename TO, int LOAD, int KW>
struct XSplit {
  static constexpr int TM = (KIND == X_DW && sizeof(T) == 2) ? 64 : 32, TN = 64, NT = 64 * KW;
  typedef XGemm<T, KIND, TM, TN, 1, 1, 1, TO, LOAD> B;   // one wave's loads, fragments and products
  static constexpr bool PN = B::PN, QN = B::QN;
  static constexpr int UP = TM / 8, UQ = TN / 8, KST = B::KST;
  static constexpr int LDS_BYTES = KW * B::STAGE;
  static_assert(TM * TN * 4 <= B::STAGE, "a partial tile fits the wave's slab");

  static __device__ inline void run(const XArgs& a, unsigned char* smem, const XTile& t) {
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int L = t.L, nk = (L + B::KB - 1) / B::KB;
    typename B::Operand P, Q;
    B::operands(a, t, P, Q);
    constexpr int NA = TM / 32;
    f32x16_t acc[NA][2];
#pragma unroll
    for (int x = 0; x < NA; ++x)
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[x][y][r] = 0.f;
    unsigned char* own = smem + wave * B::STAGE;
    typename B::frag_t fa[KST][NA], fb[KST][2];
    auto read_all = [&]() {
#pragma unroll
      for (int kk = 0; kk < KST; ++kk) B::read_frags(own, kk, 0, 0, lane, fa[kk], fb[kk]);
    };
    auto multiply = [&]() {
#pragma unroll
      for (int kk = 0; kk < KST; ++kk) B::mma(acc, fa[kk], fb[kk]);
    };
    if constexpr (LOAD == X_DIRECT) {
      const uint32_t base = lds_addr(own);
      auto issue = [&](int kt) {
        B::template dma<PN, UP>(P, kt, L, base, 0, lane);
        B::template dma<QN, UQ>(Q, kt, L, base + B::P_BYTES, 0, lane);
      };
      // Of this wave's slabs; X_FWD's column tiles begin at different ones.  They run at
      // one pace, and where the weights' pitch is a power of two, the lines of one l in all
      // rows lie in a few of the memory's channels: 64 rows, 4096 x 4096, 21.6 us without
      // this and 15.1 with it; 48 rows over 8 experts, 2048 x 5632 from HBM, 40 and 35.
      const int count = (nk - wave + KW - 1) / KW;
      int i = KIND == X_FWD && count > 0 ? t.j0 / TN % count : 0;
      auto slab_of = [&]() { return wave + i * KW; };
      if (count > 0) issue(slab_of());
      for (int left = count; left > 0; --left) {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");     // the slab is in
        read_all();
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // and in the registers
        i = i + 1 < count ? i + 1 : 0;
        if (left > 1) issue(slab_of());
        multiply();
      }
    } else {
      u32x4_t bp[UP], bq[UQ];
      const uint32_t base = lds_addr(own);
      auto fetch = [&](int kt) {
        if constexpr (!B::PD) B::template fetch<PN, UP>(P, kt, L, 0, lane, bp);
        if constexpr (!B::QD) B::template fetch<QN, UQ>(Q, kt, L, 0, lane, bq);
      };
      auto issue = [&](int kt) {
        if constexpr (B::PD) B::template dma<PN, UP>(P, kt, L, base, 0, lane);
        if constexpr (B::QD) B::template dma<QN, UQ>(Q, kt, L, base + B::P_BYTES, 0, lane);
      };
      if (wave < nk) {
        fetch(wave);
        issue(wave);
      }
      for (int kt = wave; kt < nk; kt += KW) {
        if constexpr (!B::PD) B::template put<PN, UP>(P, kt, L, bp, own, 0, lane);
        if constexpr (!B::QD) B::template put<QN, UQ>(Q, kt, L, bq, own + B::P_BYTES, 0, lane);
        if constexpr (B::PD || B::QD) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        else asm volatile("" ::: "memory");   // a wave's LDS accesses execute in order
        if (kt + KW < nk) fetch(kt + KW);
        read_all();
        if constexpr (B::PD || B::QD) asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        else asm volatile("" ::: "memory");
        if (kt + KW < nk) issue(kt + KW);
        multiply();
      }
    }
    float* part = reinterpret_cast<float*>(own);
    const int half = lane >> 5, l32 = lane & 31;
#pragma unroll
    for (int x = 0; x < NA; ++x)
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          part[(32 * x + 8 * (r >> 2) + 4 * half + (r & 3)) * TN + 32 * y + l32] = acc[x][y][r];
    __syncthreads();
    const int ncols = KIND == X_FWD ? a.m : a.k;
    TO* C = static_cast<TO*>(a.C) + (KIND == X_DW ? (static_cast<int64_t>(t.e) * a.m + t.i0) * a.ldc
                                                  : t.row0 * a.ldc);
    constexpr int EPV = 16 / sizeof(TO), PPR = TN / EPV;   // pieces of 16 bytes
    for (int p = tid; p < TM * PPR; p += NT) {
      const int i = p / PPR, jj = p % PPR * EPV, j = t.j0 + jj;
      if (i >= t.rows || j >= ncols) continue;
      f32x4_t s[EPV / 4];
#pragma unroll
      for (int v = 0; v < EPV / 4; ++v) {
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          const f32x4_t x = *reinterpret_cast<const f32x4_t*>(smem + w * B::STAGE + (i * TN + jj + 4 * v) * 4);
#pragma unroll
          for (int e = 0; e < 4; ++e) s[v][e] = w == 0 ? x[e] : s[v][e] + x[e];
        }
      }
      typedef TO out_t __attribute__((ext_vector_type(EPV)));
      out_t o;
#pragma unroll
      for (int e = 0; e < EPV; ++e) o[e] = from_f32<TO>(s[e / 4][e % 4]);
      TO* c = C + static_cast<int64_t>(i) * a.ldc + j;
      if (j + EPV <= ncols) {
        if (a.vec_out)
          *reinterpret_cast<gptr<out_t>>(global(c)) = o;
        else
          store16_loose(c, __builtin_bit_cast(u32x4_t, o));
      } else {
#pragma unroll
        for (int e = 0; e < EPV; ++e)
          if (j + e < ncols) global(c)[e] = o[e];
      }
    }
  }
};

template <typename G, int KIND>
__global__ __launch_bounds__(G::NT) void k_expert_split(XArgs a) {
  __shared__ __attribute__((aligned(1024))) unsigned char smem[G::LDS_BYTES];
  static_assert(KIND == X_DW || sizeof(XSegs) <= sizeof(smem), "segment table");
  XTile t;
  int ways;
  if (!x_tile<KIND, G::TM, G::TN, false>(a, smem, t, ways)) return;
  G::run(a, smem, t);
}

// Blocks of a launch with at most `tiles` whole tiles: cutting the last few adds fewer
// than `slots`.
inline int64_t x_blocks(int64_t tiles, bool splits, int slots) { return splits ? tiles + slots : tiles; }

}  // namespace mo
