// Host side of the row operators: mo_group_rows, mo_embedding_lookup, mo_embedding_grad.
#include "rows.h"

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "host.h"

using namespace mo;

namespace {

constexpr int64_t MAX_KEYS = int64_t(1) << 26;
constexpr int64_t MAX_ROWS = 0x7fffffffLL;
constexpr int64_t MAX_WIDTH = int64_t(1) << 24;

int key_bits(int64_t num_keys) {   // bits of the largest key, num_keys itself
  int b = 1;
  while ((int64_t(1) << b) <= num_keys) ++b;
  return b;
}

// workspace of a grouping: pairs twice (read and written by turns), the sorted keys,
// the counts and the totals
struct GroupPlan {
  int passes, bits;
  int64_t nblk;
  size_t off_pairs[2], off_keys, off_counts, off_totals, bytes;
};

GroupPlan plan_group(int64_t n, int64_t num_keys) {
  GroupPlan p = {};
  const int b = key_bits(num_keys);
  p.passes = (b + GROUP_BITS - 1) / GROUP_BITS;
  p.bits = (b + p.passes - 1) / p.passes;
  p.bits = p.bits <= 4 ? 4 : p.bits <= 7 ? 7 : p.bits;
  p.nblk = cdiv(n, GROUP_ROUNDS * 1024);
  if (n <= GROUP_ONE) return p;
  size_t off = 0;
  auto take = [&](size_t nb) {
    const size_t at = off;
    off = align_up(off + nb, ALIGN);
    return at;
  };
  const size_t rows = static_cast<size_t>(n);
  p.off_pairs[0] = take(p.passes > 1 ? rows * 8 : 0);
  p.off_pairs[1] = take(p.passes > 2 ? rows * 8 : 0);
  p.off_keys = take(p.passes > 1 ? rows * 4 : 0);
  p.off_counts = take((size_t(1) << p.bits) * static_cast<size_t>(p.nblk) * 4);
  p.off_totals = take((size_t(1) << p.bits) * 4);
  p.bytes = off;
  return p;
}

int check_keys(const char* what, const void* keys, int32_t key_bytes, int64_t n, int64_t num_keys) {
  if (key_bytes != 4 && key_bytes != 8)
    return fail(MO_ERR_UNSUPPORTED, std::string(what) + " must be 4- or 8-byte integers");
  if (n < 0 || n > MAX_ROWS) return fail(MO_ERR_INVALID, "n must be in [0, 2^31)");
  if (num_keys < 1 || num_keys > MAX_KEYS) return fail(MO_ERR_INVALID, "the number of keys must be in [1, 2^26]");
  if (n > 0 && !keys) return fail(MO_ERR_INVALID, std::string(what) + " is NULL");
  return MO_OK;
}

int check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return MO_OK;
  if (!ws) return fail(MO_ERR_WORKSPACE, "workspace is NULL");
  if (reinterpret_cast<uintptr_t>(ws) & (ALIGN - 1))
    return fail(MO_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  if (have < need) return fail(MO_ERR_WORKSPACE, "workspace too small: need " + std::to_string(need) + " bytes");
  return MO_OK;
}

template <typename F>
void with_bits(int bits, F&& f) {
  if (bits == 4) f(std::integral_constant<int, 4>{});
  else if (bits == 7) f(std::integral_constant<int, 7>{});
  else if (bits == 8) f(std::integral_constant<int, 8>{});
  else f(std::integral_constant<int, 9>{});
}

// zero: memory that the launch may clear as well, up to GROUP_ONE rows
int run_group(int pk, const KeySource& src, int64_t n, const GroupPlan& p, int32_t* order, int32_t* offsets,
              unsigned char* ws, const ZeroFill& zero, hipStream_t stream) {
  const int64_t count = static_cast<int64_t>(src.num_keys) + 1;
  if (n == 0)
    return launch(pk, stream, [&] {
      hipLaunchKernelGGL(k_group_none, dim3(cdiv(count, 256)), dim3(256), 0, stream, offsets, count);
    });
  if (n <= GROUP_ONE) {
    // blocks beyond the first only share the offsets
    const int64_t sorters = std::min<int64_t>(64, cdiv(count, 1024)), blocks = sorters + cdiv(zero.bytes, ZERO_BLOCK);
    return launch(pk, stream, [&] {
      with_bits(p.bits, [&](auto bits) {
        hipLaunchKernelGGL(k_group_small<decltype(bits)::value>, dim3(static_cast<uint32_t>(blocks)), dim3(1024), 0,
                           stream, src, static_cast<int>(n), p.passes, static_cast<int>(sorters), zero, order,
                           offsets);
      });
    });
  }
  uint32_t* counts = reinterpret_cast<uint32_t*>(ws + p.off_counts);
  uint32_t* totals = reinterpret_cast<uint32_t*>(ws + p.off_totals);
  uint32_t* keys = reinterpret_cast<uint32_t*>(ws + p.off_keys);
  uint2* pairs[2] = {reinterpret_cast<uint2*>(ws + p.off_pairs[0]), reinterpret_cast<uint2*>(ws + p.off_pairs[1])};
  const dim3 grid(p.nblk), thr(1024);
  const int nblk = static_cast<int>(p.nblk), nd = 1 << p.bits;
  const bool scan = p.nblk > GROUP_SUMS;
  const std::true_type yes;
  const std::false_type no;
  for (int d = 0; d < p.passes; ++d) {
    const uint2* in = d > 0 ? pairs[(d - 1) & 1] : nullptr;
    uint2* out = pairs[d & 1];
    const int shift = d * p.bits;
    const bool first = d == 0, last = d + 1 == p.passes;
    auto count = [&](auto f) {
      hipLaunchKernelGGL(k_group_count<decltype(f)::value>, grid, thr, 0, stream, src, in, n, shift, p.bits, counts);
    };
    auto move = [&](auto f, auto l) {
      with_bits(p.bits, [&](auto bits) {
        hipLaunchKernelGGL((k_group_move<decltype(bits)::value, decltype(f)::value, decltype(l)::value>), grid, thr,
                           0, stream, src, in, n, shift, nblk, counts, scan ? totals : nullptr, out, keys, order,
                           offsets);
      });
    };
    MO_TRY(launch(pk, stream, [&] {
      if (first) count(yes);
      else count(no);
    }));
    if (scan)
      MO_TRY(launch(pk, stream, [&] {
        hipLaunchKernelGGL(k_group_scan, dim3(cdiv(nd, 64)), dim3(64), 0, stream, counts, nblk, nd, totals);
      }));
    MO_TRY(launch(pk, stream, [&] {
      if (first && last) move(yes, yes);
      else if (first) move(yes, no);
      else if (last) move(no, yes);
      else move(no, no);
    }));
  }
  if (p.passes == 1) return MO_OK;
  return launch(pk, stream, [&] {
    hipLaunchKernelGGL(k_group_offsets, dim3(cdiv(count, 256)), dim3(256), 0, stream, keys, n, count, offsets);
  });
}

// workspace of the table's gradient: the order, the offsets, the partial sums, and the
// grouping's own
struct EmbedPlan {
  GroupPlan group;
  int64_t chunks;
  size_t off_order, off_offsets, off_partial, off_tail, off_group, bytes;
};

EmbedPlan plan_embed(int64_t n, int64_t vocab, int64_t dim) {
  EmbedPlan p = {};
  p.group = plan_group(n, vocab);
  p.chunks = cdiv(n, EG_ROWS);
  size_t off = 0;
  auto take = [&](size_t nb) {
    const size_t at = off;
    off = align_up(off + nb, ALIGN);
    return at;
  };
  p.off_order = take(static_cast<size_t>(n) * 4);
  p.off_offsets = take((static_cast<size_t>(vocab) + 1) * 4);
  p.off_partial = take(static_cast<size_t>(p.chunks) * 2 * static_cast<size_t>(round_up(dim, ROW_W)) * 4);
  p.off_tail = take(static_cast<size_t>(p.chunks) * 4);
  p.off_group = take(p.group.bytes);
  p.bytes = off;
  return p;
}

int check_embed(int64_t n, int64_t vocab, int64_t dim, int32_t dtype, int32_t out_dtype, float scale) {
  if (!valid_dtype(dtype) || !valid_dtype(out_dtype))
    return fail(MO_ERR_UNSUPPORTED, "dtypes must be MO_F32 or MO_BF16");
  if (dim < 1 || dim > MAX_WIDTH) return fail(MO_ERR_INVALID, "dim must be in [1, 2^24]");
  if (!std::isfinite(scale)) return fail(MO_ERR_INVALID, "scale must be finite");
  (void)n;
  (void)vocab;
  return MO_OK;
}

template <typename T, typename TO>
int run_embed_grad(const EmbedGrad& a, int64_t blocks, hipStream_t stream) {
  MO_TRY(launch_blocks(PK_EGRAD, stream, blocks, 256, [&](int64_t first, uint32_t count) {
    EmbedGrad b = a;
    b.first_block = first;
    if (a.dim >= ROW_W)
      hipLaunchKernelGGL((k_embed_grad<T, TO, true>), dim3(count), dim3(256), 0, stream, b);
    else
      hipLaunchKernelGGL((k_embed_grad<T, TO, false>), dim3(count), dim3(256), 0, stream, b);
  }));
  if (a.n <= EG_ROWS) return MO_OK;   // one chunk: nothing crosses
  return launch(PK_EGRAD, stream, [&] {
    const int parts = static_cast<int>(cdiv(a.dim, EJ_COLS));
    hipLaunchKernelGGL(k_embed_join<TO>, dim3(cdiv(cdiv(a.n, EG_ROWS), EJ_CHUNKS) * parts), dim3(256), 0, stream, a,
                       parts);
  });
}

}  // namespace

extern "C" {

size_t mo_group_rows_workspace_bytes(int64_t n, int64_t num_keys) {
  g_err.clear();
  if (n < 0 || n > MAX_ROWS || num_keys < 1 || num_keys > MAX_KEYS) return 0;
  return plan_group(n, num_keys).bytes;
}

int32_t mo_group_rows(const void* keys, int32_t key_bytes, int64_t n, int64_t num_keys, int32_t* order,
                      int32_t* offsets, void* workspace, size_t workspace_bytes, void* stream) {
  return entry([&]() -> int32_t {
    MO_TRY(check_keys("keys", keys, key_bytes, n, num_keys));
    if (!offsets || (n > 0 && !order)) return fail(MO_ERR_INVALID, "order or offsets is NULL");
    const GroupPlan p = plan_group(n, num_keys);
    MO_TRY(check_workspace(workspace, workspace_bytes, p.bytes));
    const ByteRows in = byte_rows(keys, 1, n, n, key_bytes);
    MO_TRY(check_apart("order", byte_rows(order, 1, n, n, 4), {in}));
    MO_TRY(check_apart("offsets", byte_rows(offsets, 1, num_keys + 1, num_keys + 1, 4), {in}));
    const KeySource src = {keys, key_bytes == 8, static_cast<uint32_t>(num_keys)};
    return run_group(PK_GROUP, src, n, p, order, offsets, static_cast<unsigned char*>(workspace),
                     ZeroFill{nullptr, 0}, static_cast<hipStream_t>(stream));
  });
}

int32_t mo_embedding_lookup(const void* table, int64_t ldt, const void* tokens, int32_t token_bytes, int64_t n,
                            int64_t vocab, int64_t dim, int32_t dtype, int32_t out_dtype, float scale, void* out,
                            void* stream_ptr) {
  return entry([&]() -> int32_t {
    MO_TRY(check_keys("tokens", tokens, token_bytes, n, vocab));
    MO_TRY(check_embed(n, vocab, dim, dtype, out_dtype, scale));
    if (ldt < dim) return fail(MO_ERR_INVALID, "table: the row pitch must be >= dim");
    if (n == 0) return MO_OK;
    if (!table || !out) return fail(MO_ERR_INVALID, "table or out is NULL");
    MO_TRY(check_apart("out", byte_rows(out, n, dim, dim, dtype_size(out_dtype)),
                       {byte_rows(table, vocab, dim, ldt, dtype_size(dtype)),
                        byte_rows(tokens, 1, n, n, token_bytes)}));
    const KeySource src = {tokens, token_bytes == 8, static_cast<uint32_t>(vocab)};
    hipStream_t stream = static_cast<hipStream_t>(stream_ptr);
    return launch_blocks(PK_LOOKUP, stream, cdiv(n, 4), 256, [&](int64_t first, uint32_t count) {
#define MO_LOOKUP_W(T, TO, W)                                                                                   \
  hipLaunchKernelGGL((k_embed_lookup<T, TO, W>), dim3(count), dim3(256), 0, stream, static_cast<const T*>(table), ldt, \
                     src, first, n, static_cast<int>(dim), scale, static_cast<TO*>(out))
#define MO_LOOKUP(T, TO)                        \
  do {                                          \
    if (dim >= ROW_W) MO_LOOKUP_W(T, TO, true); \
    else MO_LOOKUP_W(T, TO, false);             \
  } while (0)
      if (dtype == MO_F32) {
        if (out_dtype == MO_F32) MO_LOOKUP(float, float); else MO_LOOKUP(float, bf16_t);
      } else {
        if (out_dtype == MO_F32) MO_LOOKUP(bf16_t, float); else MO_LOOKUP(bf16_t, bf16_t);
      }
#undef MO_LOOKUP
#undef MO_LOOKUP_W
    });
  });
}

size_t mo_embedding_grad_workspace_bytes(int64_t n, int64_t vocab, int64_t dim) {
  g_err.clear();
  if (n < 0 || n > MAX_ROWS || vocab < 1 || vocab > MAX_KEYS || dim < 1 || dim > MAX_WIDTH) return 0;
  return plan_embed(n, vocab, dim).bytes;
}

int32_t mo_embedding_grad(const void* grad_out, int64_t ldg, const void* tokens, int32_t token_bytes, int64_t n,
                          int64_t vocab, int64_t dim, int32_t dtype, int32_t grad_dtype, float scale, void* grad,
                          void* workspace, size_t workspace_bytes, void* stream_ptr) {
  return entry([&]() -> int32_t {
    MO_TRY(check_keys("tokens", tokens, token_bytes, n, vocab));
    MO_TRY(check_embed(n, vocab, dim, dtype, grad_dtype, scale));
    if (ldg < dim) return fail(MO_ERR_INVALID, "grad_out: the row pitch must be >= dim");
    if (!grad || (n > 0 && !grad_out)) return fail(MO_ERR_INVALID, "grad_out or grad is NULL");
    const EmbedPlan p = plan_embed(n, vocab, dim);
    MO_TRY(check_workspace(workspace, workspace_bytes, p.bytes));
    MO_TRY(check_apart("grad", byte_rows(grad, vocab, dim, dim, dtype_size(grad_dtype)),
                       {byte_rows(grad_out, n, dim, ldg, dtype_size(dtype)), byte_rows(tokens, 1, n, n, token_bytes)}));
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    hipStream_t stream = static_cast<hipStream_t>(stream_ptr);
    EmbedGrad a = {};
    a.g = grad_out;
    a.ldg = ldg;
    a.order = reinterpret_cast<int32_t*>(ws + p.off_order);
    a.offsets = reinterpret_cast<int32_t*>(ws + p.off_offsets);
    a.tokens = {tokens, token_bytes == 8, static_cast<uint32_t>(vocab)};
    a.n = n;
    a.dim = static_cast<int>(dim);
    a.parts = static_cast<int>(cdiv(dim, EG_COLS));
    a.scale = scale;
    a.out = grad;
    a.partial = reinterpret_cast<float*>(ws + p.off_partial);
    a.tail_to = reinterpret_cast<int32_t*>(ws + p.off_tail);
    a.pitch = static_cast<int>(round_up(dim, ROW_W));
    a.run_blocks = cdiv(p.chunks * a.parts, 4);
    const bool zeroed = n > 0 && n <= GROUP_ONE;   // by the grouping's launch
    ZeroFill zero = {grad, 0};
    if (zeroed) zero.bytes = vocab * dim * static_cast<int64_t>(dtype_size(grad_dtype));
    const int64_t blocks = a.run_blocks + (zeroed ? 0 : cdiv(vocab, EG_ZERO));
    // a table of 2^39 bytes, and rows of 2^40 elements, are more than the device holds
    if (cdiv(zero.bytes, ZERO_BLOCK) >= (1 << 21) || cdiv(p.chunks, EJ_CHUNKS) * cdiv(dim, EJ_COLS) >= (1 << 24))
      return fail(MO_ERR_INVALID, "too many blocks for one launch");
    MO_TRY(run_group(PK_EGRAD, a.tokens, n, p.group, const_cast<int32_t*>(a.order), const_cast<int32_t*>(a.offsets),
                     ws + p.off_group, zero, stream));
    if (dtype == MO_F32) {
      if (grad_dtype == MO_F32) return run_embed_grad<float, float>(a, blocks, stream);
      return run_embed_grad<float, bf16_t>(a, blocks, stream);
    }
    if (grad_dtype == MO_F32) return run_embed_grad<bf16_t, float>(a, blocks, stream);
    return run_embed_grad<bf16_t, bf16_t>(a, blocks, stream);
  });
}

}  // extern "C"
