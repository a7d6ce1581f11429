// C ABI of the NVFP4 key/value cache and its attention (declared in
// include/nvfp4.h): argument validation on the host before any HIP call, then
// the gfx950 kernels.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <initializer_list>

#include "../../include/nvfp4.h"
#include "launchers.h"

namespace {

using nvfp4::clear_error;
using nvfp4::device_ok;

int fail(int status, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return nvfp4::set_error(status, buf);
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
hipStream_t hs(void* s) { return reinterpret_cast<hipStream_t>(s); }
int done(hipError_t e, const char* where) { return e == hipSuccess ? NVFP4_OK : nvfp4::set_hip_error(e, where); }

constexpr int64_t kMaxHeads = 65536;
constexpr int64_t kMaxSlots = ((int64_t)1 << 31) - 1;  // slots are int32
constexpr int64_t kMaxStride = (int64_t)1 << 34;  // spans of kMaxTokens rows stay below 2^63 bytes
constexpr int64_t kMaxTokens = (int64_t)1 << 27;
constexpr int64_t kMaxSequences = 65536;
constexpr int64_t kMaxRows = (int64_t)1 << 30;  // of a call of attention: numbered by int32
constexpr int64_t kMaxGroups = (int64_t)1 << 24;  // of 256 threads, half of it of 512: a launch stays below 2^32 work-items

int page_shift(int64_t page_size) {
  int s = 0;
  while (((int64_t)1 << s) < page_size) ++s;
  return s;
}

bool cache_sizes_ok(int64_t heads, int64_t head_dim, int64_t page_size) {
  return heads > 0 && heads <= kMaxHeads && (head_dim == 64 || head_dim == 128 || head_dim == 256) && page_size >= 32 &&
         page_size <= 65536 && (page_size & (page_size - 1)) == 0;
}

int check_cache(const void* cache, int64_t pages, int64_t page_size, int64_t heads, int64_t head_dim,
                const float* k_scale, const float* v_scale) {
  if (pages < 0 || heads <= 0) return fail(NVFP4_ERR_INVALID_VALUE, "pages=%lld, heads=%lld", (long long)pages, (long long)heads);
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "head_dim=%lld: 64, 128 or 256", (long long)head_dim);
  if (!cache_sizes_ok(heads, head_dim, page_size))
    return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "page_size=%lld: a power of two, 32 .. 65536; heads=%lld: at most %lld",
                (long long)page_size, (long long)heads, (long long)kMaxHeads);
  if (pages > kMaxSlots / page_size)
    return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%lld pages of %lld tokens: at most 2^31 - 1 slots", (long long)pages,
                (long long)page_size);
  if ((pages > 0 && !cache) || !k_scale || !v_scale)
    return fail(NVFP4_ERR_INVALID_VALUE, "cache, k_scale and v_scale are required");
  if (!aligned(cache, 16) || !aligned(k_scale, 4) || !aligned(v_scale, 4))
    return fail(NVFP4_ERR_MISALIGNED, "cache must be 16-byte aligned, k_scale and v_scale 4-byte aligned");
  return NVFP4_OK;
}

// A [tokens, width] bf16 argument whose rows start `stride` elements apart.
int check_rows(const void* p, int64_t stride, int64_t width, const char* name) {
  if (!p) return fail(NVFP4_ERR_INVALID_VALUE, "%s is required", name);
  if (stride < width || stride > kMaxStride)
    return fail(NVFP4_ERR_INVALID_VALUE, "%s's stride %lld: at least its %lld elements, at most 2^34", name,
                (long long)stride, (long long)width);
  if (stride % 8 != 0 || !aligned(p, 16))
    return fail(NVFP4_ERR_MISALIGNED, "%s must be 16-byte aligned, its stride a multiple of 8", name);
  return NVFP4_OK;
}

// A buffer of a call: `rows` pieces of `width` bytes, `stride` bytes apart.
struct Buffer {
  const void* p;
  int64_t rows, width, stride;
  const char* name;
};

Buffer whole(const void* p, int64_t bytes, const char* name) { return {p, 1, bytes, bytes, name}; }

bool overlap(const Buffer& a, const Buffer& b) {
  if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
  const int64_t d = (int64_t)(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p));
  if (d >= (a.rows - 1) * a.stride + a.width || d <= -((b.rows - 1) * b.stride + b.width)) return false;
  if (a.stride != b.stride || a.rows != b.rows) return true;  // their spans meet
  // columns of one matrix: row j of b lies d + (j - i) stride after row i of a
  int64_t n = d / a.stride;
  for (int64_t shift = -n - 1; shift <= -n + 1; ++shift) {
    const int64_t at = d + shift * a.stride;
    if (shift > -a.rows && shift < a.rows && at < a.width && at > -b.width) return true;
  }
  return false;
}

int check_outputs(std::initializer_list<Buffer> outputs, std::initializer_list<Buffer> inputs) {
  for (const Buffer* o = outputs.begin(); o != outputs.end(); ++o) {
    for (const Buffer& i : inputs)
      if (overlap(*o, i)) return fail(NVFP4_ERR_INVALID_VALUE, "%s overlaps %s", o->name, i.name);
    for (const Buffer* p = outputs.begin(); p != o; ++p)
      if (overlap(*o, *p)) return fail(NVFP4_ERR_INVALID_VALUE, "%s overlaps %s", o->name, p->name);
  }
  return NVFP4_OK;
}

int check_tokens(int64_t tokens) {
  if (tokens < 0) return fail(NVFP4_ERR_INVALID_VALUE, "tokens=%lld", (long long)tokens);
  if (tokens > kMaxTokens) return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "tokens=%lld: at most 2^27", (long long)tokens);
  return NVFP4_OK;
}

bool attention_sizes_ok(int64_t sequences, int64_t tokens, int64_t q_heads, int64_t heads, int64_t head_dim,
                        int64_t page_size, int64_t table_pages, int64_t window, int one_each) {
  return sequences > 0 && sequences <= kMaxSequences && tokens > 0 && tokens <= kMaxTokens && table_pages > 0 &&
         cache_sizes_ok(heads, head_dim, page_size) && table_pages <= kMaxSlots / page_size && q_heads > 0 &&
         q_heads <= kMaxHeads && q_heads % heads == 0 && window >= 0 && tokens * q_heads <= kMaxRows &&
         (!one_each || sequences == tokens);
}

int64_t page_bytes(int64_t heads, int64_t head_dim, int64_t page_size) { return heads * (page_size / 32) * 36 * head_dim; }

}  // namespace

extern "C" {

NVFP4_API size_t nvfp4_kv_page_bytes(int64_t heads, int64_t head_dim, int64_t page_size) {
  return cache_sizes_ok(heads, head_dim, page_size) ? (size_t)page_bytes(heads, head_dim, page_size) : 0;
}

NVFP4_API int nvfp4_kv_append(const void* k, int64_t k_stride, const void* v, int64_t v_stride, const void* q,
                              int64_t q_stride, void* q_out, int64_t q_out_stride, int64_t q_heads,
                              const int32_t* positions, const float* rope, int64_t max_positions, int64_t rope_dim,
                              int interleaved, const int32_t* slots, int64_t tokens, uint8_t* cache, int64_t pages,
                              int64_t page_size, int64_t heads, int64_t head_dim, const float* k_scale,
                              const float* v_scale, void* stream) {
  clear_error();
  int st = check_tokens(tokens);
  if (st || (st = check_cache(cache, pages, page_size, heads, head_dim, k_scale, v_scale))) return st;
  if ((q == nullptr) != (q_out == nullptr) && tokens > 0)
    return fail(NVFP4_ERR_INVALID_VALUE, "q and q_out go together");
  if (q && (q_heads <= 0 || q_heads > kMaxHeads))
    return fail(NVFP4_ERR_INVALID_VALUE, "q_heads=%lld: 1 .. %lld", (long long)q_heads, (long long)kMaxHeads);
  if (rope_dim < 0 || rope_dim > head_dim || rope_dim % 32 != 0)
    return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "rope_dim=%lld: a multiple of 32 up to head_dim", (long long)rope_dim);
  if (tokens == 0) return NVFP4_OK;
  if (rope_dim > 0 && (max_positions <= 0 || max_positions > kMaxSlots))
    return fail(NVFP4_ERR_INVALID_VALUE, "max_positions=%lld: 1 .. 2^31 - 1", (long long)max_positions);
  const int64_t kw = heads * head_dim, qw = q ? q_heads * head_dim : 0;
  if ((st = check_rows(k, k_stride, kw, "k")) || (st = check_rows(v, v_stride, kw, "v"))) return st;
  if (q && ((st = check_rows(q, q_stride, qw, "q")) || (st = check_rows(q_out, q_out_stride, qw, "q_out")))) return st;
  if (!slots) return fail(NVFP4_ERR_INVALID_VALUE, "slots are required");
  if (!aligned(slots, 4)) return fail(NVFP4_ERR_MISALIGNED, "slots must be 4-byte aligned");
  if (rope_dim > 0) {
    if (!positions || !rope) return fail(NVFP4_ERR_INVALID_VALUE, "positions and rope are required with rope_dim > 0");
    if (!aligned(positions, 4) || !aligned(rope, 16))
      return fail(NVFP4_ERR_MISALIGNED, "positions must be 4-byte aligned, rope 16-byte aligned");
  }
  if (nvfp4::kv_append_workgroups(tokens, q ? q_heads : 0, heads, (int)head_dim) >= kMaxGroups)
    return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%lld tokens of %lld + %lld heads in one call", (long long)tokens,
                (long long)q_heads, (long long)heads);
  const Buffer bk = {k, tokens, 2 * kw, 2 * k_stride, "k"}, bv = {v, tokens, 2 * kw, 2 * v_stride, "v"},
               bq = {q, tokens, 2 * qw, 2 * q_stride, "q"}, bo = {q_out, tokens, 2 * qw, 2 * q_out_stride, "q_out"},
               bc = whole(cache, pages * page_bytes(heads, head_dim, page_size), "cache"),
               bs = whole(slots, 4 * tokens, "slots"),
               bp = whole(rope_dim ? positions : nullptr, 4 * tokens, "positions"),
               br = whole(rope_dim ? rope : nullptr, 4 * max_positions * rope_dim, "rope"),
               b1 = whole(k_scale, 4 * heads, "k_scale"), b2 = whole(v_scale, 4 * heads, "v_scale");
  if ((st = check_outputs({bc, bo}, {bk, bv, bs, bp, br, b1, b2}))) return st;
  if (overlap(bc, bq)) return fail(NVFP4_ERR_INVALID_VALUE, "cache overlaps q");
  if (!(q_out == q && q_out_stride == q_stride) && overlap(bo, bq))
    return fail(NVFP4_ERR_INVALID_VALUE, "q_out overlaps q at another place or stride");
  if ((st = device_ok())) return st;
  nvfp4::KvAppend a = {};
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.q = static_cast<const uint16_t*>(q);
  a.q_out = static_cast<uint16_t*>(q_out);
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_stride = q_stride;
  a.q_out_stride = q_out_stride;
  a.slots = slots;
  a.positions = positions;
  a.rope = rope;
  a.cache = cache;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.tokens = (int)tokens;
  a.q_heads = q ? (int)q_heads : 0;
  a.heads = (int)heads;
  a.rot = (int)rope_dim;
  a.max_positions = rope_dim ? (int)max_positions : 0;
  a.interleaved = interleaved;
  a.page_shift = page_shift(page_size);
  a.slot_limit = (int)(pages * page_size);
  return done(nvfp4::launch_kv_append(a, (int)head_dim, hs(stream)), "kv_append launch");
}

NVFP4_API int nvfp4_kv_read(const uint8_t* cache, int64_t pages, int64_t page_size, int64_t heads, int64_t head_dim,
                            const float* k_scale, const float* v_scale, const int32_t* slots, int64_t tokens, void* k,
                            void* v, int out_dtype, void* stream) {
  clear_error();
  int st = check_tokens(tokens);
  if (st || (st = check_cache(cache, pages, page_size, heads, head_dim, k_scale, v_scale))) return st;
  if (out_dtype != NVFP4_BF16 && out_dtype != NVFP4_F32) return fail(NVFP4_ERR_INVALID_VALUE, "out_dtype %d", out_dtype);
  if (tokens == 0) return NVFP4_OK;
  if (!slots || !k || !v) return fail(NVFP4_ERR_INVALID_VALUE, "slots, k and v are required");
  if (!aligned(slots, 4) || !aligned(k, 16) || !aligned(v, 16))
    return fail(NVFP4_ERR_MISALIGNED, "k and v must be 16-byte aligned, slots 4-byte aligned");
  if (nvfp4::kv_read_workgroups(tokens, heads, (int)head_dim, out_dtype == NVFP4_F32) >= kMaxGroups)
    return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%lld tokens of %lld heads in one call", (long long)tokens, (long long)heads);
  const int64_t bytes = tokens * heads * head_dim * (out_dtype == NVFP4_F32 ? 4 : 2);
  if ((st = check_outputs({whole(k, bytes, "k"), whole(v, bytes, "v")},
                          {whole(cache, pages * page_bytes(heads, head_dim, page_size), "cache"),
                           whole(slots, 4 * tokens, "slots"), whole(k_scale, 4 * heads, "k_scale"),
                           whole(v_scale, 4 * heads, "v_scale")})))
    return st;
  if ((st = device_ok())) return st;
  const nvfp4::KvRead a = {cache, k_scale, v_scale, slots, k, v, (int)tokens, (int)heads, page_shift(page_size),
                           (int)(pages * page_size)};
  return done(nvfp4::launch_kv_read(a, (int)head_dim, out_dtype == NVFP4_F32, hs(stream)), "kv_read launch");
}

NVFP4_API size_t nvfp4_kv_attention_workspace_size(int64_t sequences, int64_t tokens, int64_t q_heads, int64_t heads,
                                                   int64_t head_dim, int64_t page_size, int64_t table_pages,
                                                   int64_t window, int one_each) {
  if (!attention_sizes_ok(sequences, tokens, q_heads, heads, head_dim, page_size, table_pages, window, one_each)) return 0;
  return nvfp4::plan_kv_attention(sequences, tokens, q_heads, heads, (int)head_dim, table_pages * page_size, window,
                                  one_each != 0)
      .ws_bytes;
}

NVFP4_API int nvfp4_kv_attention_path(int64_t sequences, int64_t tokens, int64_t q_heads, int64_t heads,
                                      int64_t head_dim, int64_t page_size, int64_t table_pages, int64_t window,
                                      int one_each) {
  if (!attention_sizes_ok(sequences, tokens, q_heads, heads, head_dim, page_size, table_pages, window, one_each))
    return -1;
  return nvfp4::kv_block_rows(nvfp4::plan_kv_attention(sequences, tokens, q_heads, heads, (int)head_dim,
                                                       table_pages * page_size, window, one_each != 0),
                              (int)head_dim);
}

NVFP4_API int nvfp4_kv_attention(const void* q, int64_t q_stride, const uint8_t* cache, int64_t pages,
                                 int64_t page_size, int64_t heads, int64_t head_dim, const float* k_scale,
                                 const float* v_scale, const int32_t* page_table, int64_t table_pages,
                                 const int32_t* kv_lens, const int32_t* q_starts, int64_t sequences, int64_t tokens,
                                 int64_t q_heads, float scale, int causal, int64_t window, void* out, float* lse,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  int st = check_tokens(tokens);
  if (st || (st = check_cache(cache, pages, page_size, heads, head_dim, k_scale, v_scale))) return st;
  if (sequences < 0 || sequences > kMaxSequences)
    return fail(NVFP4_ERR_INVALID_VALUE, "sequences=%lld: 0 .. %lld", (long long)sequences, (long long)kMaxSequences);
  if (q_heads <= 0 || q_heads > kMaxHeads || q_heads % heads != 0)
    return fail(NVFP4_ERR_INVALID_VALUE, "q_heads=%lld: a multiple of heads=%lld, at most %lld", (long long)q_heads,
                (long long)heads, (long long)kMaxHeads);
  if (!std::isfinite(scale)) return fail(NVFP4_ERR_INVALID_VALUE, "scale must be finite");
  if (window < 0 || (window > 0 && !causal))
    return fail(NVFP4_ERR_INVALID_VALUE, "window=%lld: >= 0, and 0 without causal", (long long)window);
  if (table_pages < 0 || table_pages > kMaxSlots / page_size)
    return fail(NVFP4_ERR_INVALID_VALUE, "table_pages=%lld: >= 0, at most 2^31 - 1 tokens", (long long)table_pages);
  if (!q_starts && tokens != sequences)
    return fail(NVFP4_ERR_INVALID_VALUE, "without q_starts each sequence has one token: %lld tokens, %lld sequences",
                (long long)tokens, (long long)sequences);
  if (tokens * q_heads > kMaxRows)
    return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%lld tokens of %lld query heads in one call", (long long)tokens,
                (long long)q_heads);
  if (tokens == 0 || sequences == 0) return NVFP4_OK;
  if ((st = check_rows(q, q_stride, q_heads * head_dim, "q"))) return st;
  if (!kv_lens || !out || (table_pages > 0 && !page_table))
    return fail(NVFP4_ERR_INVALID_VALUE, "page_table, kv_lens and out are required");
  if (!aligned(out, 16) || !aligned(page_table, 4) || !aligned(kv_lens, 4) || !aligned(q_starts, 4) || !aligned(lse, 4))
    return fail(NVFP4_ERR_MISALIGNED, "out must be 16-byte aligned, page_table, kv_lens, q_starts and lse 4-byte aligned");
  if (pages == 0 && table_pages > 0) return fail(NVFP4_ERR_INVALID_VALUE, "a page table without pages");
  const nvfp4::KvPlan plan = nvfp4::plan_kv_attention(sequences, tokens, q_heads, heads, (int)head_dim,
                                                      table_pages * page_size, window, q_starts == nullptr);
  if ((plan.blocks + plan.parts) * heads >= (plan.tiles ? kMaxGroups : kMaxGroups / 2))
    return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%lld tokens of %lld heads in one call", (long long)tokens,
                (long long)q_heads);
  if (plan.ws_bytes > 0) {
    if (workspace_bytes < plan.ws_bytes)
      return fail(NVFP4_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes < %zu required", workspace_bytes, plan.ws_bytes);
    if (!workspace) return fail(NVFP4_ERR_INVALID_VALUE, "workspace is NULL");
    if (!aligned(workspace, 16)) return fail(NVFP4_ERR_MISALIGNED, "workspace must be 16-byte aligned");
  }
  const int64_t qw = 2 * q_heads * head_dim;
  if ((st = check_outputs({whole(out, tokens * qw, "out"), whole(lse, 4 * tokens * q_heads, "lse"),
                           whole(plan.ws_bytes ? workspace : nullptr, (int64_t)plan.ws_bytes, "workspace")},
                          {{q, tokens, qw, 2 * q_stride, "q"},
                           whole(cache, pages * page_bytes(heads, head_dim, page_size), "cache"),
                           whole(page_table, 4 * sequences * table_pages, "page_table"),
                           whole(kv_lens, 4 * sequences, "kv_lens"), whole(q_starts, 4 * (sequences + 1), "q_starts"),
                           whole(k_scale, 4 * heads, "k_scale"), whole(v_scale, 4 * heads, "v_scale")})))
    return st;
  if ((st = device_ok())) return st;
  nvfp4::KvAttend a = {};
  a.q = static_cast<const uint16_t*>(q);
  a.q_stride = q_stride;
  a.cache = cache;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.table = page_table;
  a.lens = kv_lens;
  a.starts = q_starts;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.table_pages = (int)table_pages;
  a.sequences = (int)sequences;
  a.tokens = (int)tokens;
  a.heads = (int)heads;
  a.group = (int)(q_heads / heads);
  a.pages = (int)pages;
  a.page_shift = page_shift(page_size);
  a.causal = causal != 0;
  a.window = (int)(window < kMaxSlots ? window : 0);  // a window past every context is none
  a.scale = scale;
  return done(nvfp4::launch_kv_attention(a, (int)head_dim, plan, workspace, hs(stream)), "kv_attention launch");
}

}  // extern "C"
