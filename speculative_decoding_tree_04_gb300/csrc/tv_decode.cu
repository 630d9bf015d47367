// tv_decode.cu -- argument checks of the decode cycle's calls (tv_rope, tv_norm_rope,
// tv_shared_attn, tv_token_sample; include/tv.h).
#include <cuda_runtime.h>

#include <cmath>
#include <cstdio>

#include "tv.h"
#include "tv_internal.h"

namespace {

int refuse(int code, const char* who, const char* what) {
  char buf[256];
  snprintf(buf, sizeof(buf), "%s: %s", who, what);
  tv::set_last_error(buf);
  return code;
}
int result(cudaError_t e, const char* who) {
  return e == cudaSuccess ? TV_OK : refuse(TV_ERR_CUDA, who, cudaGetErrorString(e));
}

bool aligned(const void* p, uintptr_t n) { return (uintptr_t)p % n == 0; }
bool type_ok(tv_dtype t) { return t == TV_F32 || t == TV_BF16; }
int64_t size_of(tv_dtype t) { return t == TV_BF16 ? 2 : 4; }

// Whether two arrays of the given bytes share memory (a null one does not).
bool overlap(const void* a, int64_t an, const void* b, int64_t bn) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return a && b && an > 0 && bn > 0 && x < y + (uintptr_t)bn && y < x + (uintptr_t)an;
}

// Strides of [tokens, heads] vectors of d elements whose vectors do not overlap.
bool apart(int64_t token, int64_t head, int64_t T, int64_t H, int64_t d) {
  constexpr int64_t kMost = 1ll << 31;
  if (token < 0 || head < 0 || token >= kMost || head >= kMost) return false;
  const bool by_token = (H == 1 || head >= d) && (T == 1 || token >= (H - 1) * head + d);
  const bool by_head = (T == 1 || token >= d) && (H == 1 || head >= (T - 1) * token + d);
  return by_token || by_head;
}
int64_t span(int64_t token, int64_t head, int64_t T, int64_t H, int64_t d) {
  return (T - 1) * token + (H - 1) * head + d;
}

// [T, H] vectors of d elements, `token` and `head` elements apart.
struct Vectors {
  int64_t token, head, d;
};
// Whether two such sets of one element type that start `off` elements apart share memory.  Slices of
// one buffer mostly lie between one another's vectors: those of the same strides are told exactly,
// others by the place in a stride's period that each keeps to (nothing else is: it counts as shared).
bool meet(Vectors a, Vectors b, int64_t off, int64_t T, int64_t H) {
  if (T == 1) a.token = b.token = 0;  // (a dimension of one has no stride)
  if (H == 1) a.head = b.head = 0;
  if (off >= span(a.token, a.head, T, H, a.d) || -off >= span(b.token, b.head, T, H, b.d)) return false;
  if (a.token == b.token && a.head == b.head) {
    // some differences dt and dh of the tokens and heads put b's vector within a's
    for (int64_t dh = 1 - H; dh < H; ++dh) {
      const int64_t at = off + dh * a.head;
      int64_t dt = a.token > 0 ? (a.d - 1 - at) / a.token : 0;  // the largest one not behind a's end,
      if (a.token > 0 && at + dt * a.token >= a.d) --dt;        // (division rounds to zero)
      if (dt > T - 1) dt = T - 1;
      if (dt > -T && at + dt * a.token < a.d && at + dt * a.token > -b.d) return true;
    }
    return false;
  }
  // multiples of m put aside, a lies in [0, an) and b in [at, at + bn)
  auto apart_by = [&](int64_t m, int64_t an, int64_t bn) {
    const int64_t at = (off % m + m) % m;
    return at >= an && at + bn <= m;
  };
  for (const int64_t m : {a.token, b.token})
    if (m > 0 && a.token % m == 0 && b.token % m == 0 &&
        apart_by(m, (H - 1) * a.head + a.d, (H - 1) * b.head + b.d))
      return false;
  for (const int64_t m : {a.head, b.head})
    if (m > 0 && a.head % m == 0 && b.head % m == 0 &&
        apart_by(m, (T - 1) * a.token + a.d, (T - 1) * b.token + b.d))
      return false;
  return true;
}

int check_scaling(const tv_rope_scaling* s, int rot_dim, const char* who) {
  if (!s) return refuse(TV_ERR_INVALID_ARG, who, "scaling is NULL");
  if (rot_dim < 2 || rot_dim > 512 || rot_dim % 2)
    return refuse(TV_ERR_INVALID_ARG, who, "rot_dim must be even, 2 to 512");
  if (s->kind < TV_ROPE_PLAIN || s->kind > TV_ROPE_WAVELENGTH)
    return refuse(TV_ERR_INVALID_ARG, who, "bad scaling kind");
  if (!(s->base > 1.0) || std::isinf(s->base) || !std::isfinite(s->magnitude))
    return refuse(TV_ERR_INVALID_ARG, who, "bad rope base or magnitude");
  if (s->kind != TV_ROPE_PLAIN && (!(s->factor >= 1.0) || std::isinf(s->factor)))
    return refuse(TV_ERR_INVALID_ARG, who, "scaling factor below 1");
  if (s->kind == TV_ROPE_YARN || s->kind == TV_ROPE_WAVELENGTH)
    if (!(s->original_context > 0.0) || std::isinf(s->original_context) || !(s->low > 0.0) ||
        !(s->high > s->low) || std::isinf(s->high))
      return refuse(TV_ERR_INVALID_ARG, who, "bad original_context, low or high");
  return TV_OK;
}

int check_rope(const tv_rope_args* a) {
  const char* who = "tv_rope";
  if (!a) return refuse(TV_ERR_INVALID_ARG, who, "args is NULL");
  if (a->struct_size != sizeof(tv_rope_args))
    return refuse(TV_ERR_INVALID_ARG, who, "struct_size mismatch (ABI)");
  if (a->T < 0 || a->n_heads < 1 || a->d_head < 2 || a->rot_offset < 0)
    return refuse(TV_ERR_INVALID_ARG, who, "bad T, n_heads, d_head or rot_offset");
  const int rc = check_scaling(&a->scaling, a->rot_dim, who);
  if (rc != TV_OK) return rc;
  if (a->d_head > 65536 || a->n_heads > 65536)
    return refuse(TV_ERR_UNSUPPORTED, who, "d_head and n_heads of at most 65536");
  if ((int64_t)a->rot_offset + a->rot_dim > a->d_head)
    return refuse(TV_ERR_INVALID_ARG, who, "the rotated part ends past the head");
  if (a->layout != TV_ROPE_HALF && a->layout != TV_ROPE_INTERLEAVED)
    return refuse(TV_ERR_INVALID_ARG, who, "bad layout");
  if (a->inverse != 0 && a->inverse != 1) return refuse(TV_ERR_INVALID_ARG, who, "bad inverse");
  if (!type_ok(a->dt)) return refuse(TV_ERR_INVALID_ARG, who, "bad dtype");
  if (a->T == 0) return TV_OK;
  if (!a->in || !a->out || !a->positions) return refuse(TV_ERR_INVALID_ARG, who, "NULL pointer");
  const int64_t es = size_of(a->dt), T = a->T, H = a->n_heads, d = a->d_head;
  if (!aligned(a->in, es) || !aligned(a->out, es))
    return refuse(TV_ERR_INVALID_ARG, who, "tensors not aligned to their element size");
  if (a->in_stride_token < 0 || a->in_stride_head < 0 || a->in_stride_token >= (1ll << 31) ||
      a->in_stride_head >= (1ll << 31) ||
      !apart(a->out_stride_token, a->out_stride_head, T, H, d))
    return refuse(TV_ERR_INVALID_ARG, who, "bad strides, or output heads that overlap");
  if (a->in == a->out) {
    if ((T > 1 && a->in_stride_token != a->out_stride_token) ||
        (H > 1 && a->in_stride_head != a->out_stride_head))
      return refuse(TV_ERR_INVALID_ARG, who, "in place needs equal strides");
  } else if (meet({a->in_stride_token, a->in_stride_head, d}, {a->out_stride_token, a->out_stride_head, d},
                  ((intptr_t)a->out - (intptr_t)a->in) / es, T, H)) {
    return refuse(TV_ERR_INVALID_ARG, who, "out overlaps in");
  }
  const int64_t n_out = span(a->out_stride_token, a->out_stride_head, T, H, d) * es;
  if (overlap(a->out, n_out, a->positions, 4 * T))
    return refuse(TV_ERR_INVALID_ARG, who, "out overlaps positions");
  return TV_OK;
}

int check_norm_rope(const tv_norm_rope_args* a) {
  const char* who = "tv_norm_rope";
  if (!a) return refuse(TV_ERR_INVALID_ARG, who, "args is NULL");
  if (a->struct_size != sizeof(tv_norm_rope_args))
    return refuse(TV_ERR_INVALID_ARG, who, "struct_size mismatch (ABI)");
  if (a->B < 0 || a->T < 0 || a->H < 1 || a->d_nope < 0 || a->d_rope < 2 || a->d_latent < 1)
    return refuse(TV_ERR_INVALID_ARG, who, "bad B, T, H, d_nope, d_rope or d_latent");
  const int rc = check_scaling(&a->scaling, a->rot_dim, who);
  if (rc != TV_OK) return rc;
  if (a->rot_dim > a->d_rope) return refuse(TV_ERR_INVALID_ARG, who, "rot_dim exceeds d_rope");
  if ((int64_t)a->d_nope + a->d_rope > 65536 || (int64_t)a->d_latent + a->d_rope > 65536 ||
      a->H > 65536)
    return refuse(TV_ERR_UNSUPPORTED, who, "rows, heads of at most 65536");
  if (a->layout != TV_ROPE_HALF && a->layout != TV_ROPE_INTERLEAVED)
    return refuse(TV_ERR_INVALID_ARG, who, "bad layout");
  if (!type_ok(a->dt)) return refuse(TV_ERR_INVALID_ARG, who, "bad dtype");
  if (!(a->eps >= 0.f) || std::isinf(a->eps)) return refuse(TV_ERR_INVALID_ARG, who, "bad eps");
  if (a->B == 0 || a->T == 0) return TV_OK;
  if (!a->q && !a->kv) return refuse(TV_ERR_INVALID_ARG, who, "neither q nor kv");
  if (!a->q_start || !a->prefix_len) return refuse(TV_ERR_INVALID_ARG, who, "NULL pointer");
  const int64_t es = size_of(a->dt), T = a->T, H = a->H;
  constexpr int64_t kMost = 1ll << 31;
  const void *outs[4], *ins[9];
  int64_t n_outs[4], n_ins[9];
  int o = 0, i = 0;
  auto out = [&](const void* p, int64_t n) { outs[o] = p, n_outs[o++] = n * es; };
  auto in = [&](const void* p, int64_t n) { ins[i] = p, n_ins[i++] = n; };
  in(a->q_start, 4 * ((int64_t)a->B + 1));
  in(a->prefix_len, 4ll * a->B);
  in(a->depth, 4 * T);
  if (a->q) {
    const int64_t d = (int64_t)a->d_nope + a->d_rope;
    if (!a->q_pe || (a->d_nope > 0 && !a->q_nope))
      return refuse(TV_ERR_INVALID_ARG, who, "NULL query output");
    if (a->q_stride_token < 0 || a->q_stride_head < 0 || a->q_stride_token >= kMost ||
        a->q_stride_head >= kMost)
      return refuse(TV_ERR_INVALID_ARG, who, "bad query strides");
    in(a->q, span(a->q_stride_token, a->q_stride_head, T, H, d) * es);
    in(a->q_weight, d * es);
    if (a->d_nope > 0) out(a->q_nope, T * H * a->d_nope);
    out(a->q_pe, T * H * a->d_rope);
  }
  if (a->kv) {
    const tv_cache_layout& c = a->cache;
    if (!a->c_kv || !a->k_pe) return refuse(TV_ERR_INVALID_ARG, who, "NULL cache");
    if (a->kv_stride_token < 0 || a->kv_stride_token >= kMost || a->ckv_row_stride < a->d_latent ||
        a->ckv_row_stride >= kMost || a->kpe_row_stride < a->d_rope || a->kpe_row_stride >= kMost)
      return refuse(TV_ERR_INVALID_ARG, who, "bad key or cache strides");
    if (c.num_rows <= 0 || c.num_rows >= (1ll << 40))
      return refuse(TV_ERR_INVALID_ARG, who, "cache.num_rows is required");
    if (c.page_table ? (c.page_size < 1 || c.max_pages < 1) : c.kv_stride_b < 1)
      return refuse(TV_ERR_INVALID_ARG, who, "bad cache layout");
    in(a->kv, ((T - 1) * a->kv_stride_token + a->d_latent + a->d_rope) * es);
    in(a->kv_weight, a->d_latent * es);
    in(a->k_weight, a->d_rope * es);
    in(c.page_table, 4ll * a->B * c.max_pages);
    out(a->c_kv, (c.num_rows - 1) * a->ckv_row_stride + a->d_latent);
    out(a->k_pe, (c.num_rows - 1) * a->kpe_row_stride + a->d_rope);
  }
  const int n_query = a->q ? (a->d_nope > 0 ? 2 : 1) : 0;
  for (int x = 0; x < o; ++x) {
    if (!aligned(outs[x], es)) return refuse(TV_ERR_INVALID_ARG, who, "misaligned output");
    for (int y = 0; y < i; ++y)
      if (overlap(outs[x], n_outs[x], ins[y], n_ins[y]))
        return refuse(TV_ERR_INVALID_ARG, who, "an output overlaps an input");
    for (int y = 0; y < x; ++y)
      if (y < n_query && overlap(outs[x], n_outs[x], outs[y], n_outs[y]))
        return refuse(TV_ERR_INVALID_ARG, who, "two outputs overlap");
  }
  // (the cache's two arrays may be slices of one: each with the other's rows between its own)
  if (a->kv && meet({a->ckv_row_stride, 0, a->d_latent}, {a->kpe_row_stride, 0, a->d_rope},
                    ((intptr_t)a->k_pe - (intptr_t)a->c_kv) / es, a->cache.num_rows, 1))
    return refuse(TV_ERR_INVALID_ARG, who, "c_kv and k_pe overlap");
  if (!aligned(a->q, es) || !aligned(a->kv, es) || !aligned(a->q_weight, es) ||
      !aligned(a->kv_weight, es) || !aligned(a->k_weight, es))
    return refuse(TV_ERR_INVALID_ARG, who, "tensors not aligned to their element size");
  return TV_OK;
}

int check_shared(const tv_shared_args* a) {
  const char* who = "tv_shared_attn";
  if (!a) return refuse(TV_ERR_INVALID_ARG, who, "args is NULL");
  if (a->struct_size != sizeof(tv_shared_args))
    return refuse(TV_ERR_INVALID_ARG, who, "struct_size mismatch (ABI)");
  if (a->B < 0 || a->H < 1 || a->Q < 1 || a->max_prefix_len < 0 || a->G < 0 || a->G > a->B)
    return refuse(TV_ERR_INVALID_ARG, who, "bad B, H, Q, max_prefix_len or G");
  if (!(a->scale > 0.f) || a->scale > 1e30f)
    return refuse(TV_ERR_INVALID_ARG, who, "scale must be positive");
  if (!type_ok(a->out_dt)) return refuse(TV_ERR_INVALID_ARG, who, "bad out_dt");
  if (a->dt != TV_BF16) return refuse(TV_ERR_UNSUPPORTED, who, "bf16 queries and cache only");
  if (a->d_latent != 512 || a->d_rope != 64)
    return refuse(TV_ERR_UNSUPPORTED, who, "needs d_latent 512 and d_rope 64");
  if (a->Q > 64) return refuse(TV_ERR_UNSUPPORTED, who, "Q > 64 not supported");
  const int64_t R = (int64_t)a->Q * a->H;
  if (R > (1 << 20) || a->B * (R + 128) >= (1ll << 30))
    return refuse(TV_ERR_UNSUPPORTED, who, "B * Q * H must be below 2^30");
  if (a->max_prefix_len > (1 << 30))
    return refuse(TV_ERR_UNSUPPORTED, who, "max_prefix_len of at most 2^30");
  if (a->B == 0) return TV_OK;
  if (!a->q_latent || !a->q_pe || !a->c_kv || !a->k_pe || !a->prefix_len || !a->out ||
      (a->G > 0 && (!a->group_start || !a->shared_len)))
    return refuse(TV_ERR_INVALID_ARG, who, "NULL pointer");
  const tv_cache_layout& c = a->cache;
  if (c.num_rows <= 0 || c.num_rows >= (1ll << 31) - 64)
    return refuse(TV_ERR_INVALID_ARG, who, "cache.num_rows is required, below 2^31");
  if (a->ckv_row_stride < 512 || a->kpe_row_stride < 64 || a->ckv_row_stride >= (1ll << 31) ||
      a->kpe_row_stride >= (1ll << 31) || a->ckv_row_stride % 8 || a->kpe_row_stride % 8 ||
      !aligned(a->c_kv, 16) || !aligned(a->k_pe, 16) || !aligned(a->q_latent, 16) ||
      !aligned(a->q_pe, 16) || !aligned(a->out, 32) || !aligned(a->lse, 4))
    return refuse(TV_ERR_INVALID_ARG, who, "tensors and cache rows must be 16-byte aligned (out: 32)");
  if (c.page_table) {
    if (c.page_size != 64) return refuse(TV_ERR_UNSUPPORTED, who, "needs 64-token pages");
    if (c.max_pages < 1 || (int64_t)c.max_pages * 64 >= (1ll << 31))
      return refuse(TV_ERR_INVALID_ARG, who, "bad max_pages");
  } else if (c.kv_stride_b < 1 || c.kv_stride_b >= (1ll << 31) || (int64_t)a->B * c.kv_stride_b > c.num_rows) {
    return refuse(TV_ERR_INVALID_ARG, who, "kv_stride_b outside 1 .. num_rows / B");
  }
  const int64_t n = a->B * R, es = size_of(a->out_dt);
  const struct {
    const void* p;
    int64_t n;
  } ins[8] = {{a->q_latent, n * 1024},
              {a->q_pe, n * 128},
              {a->c_kv, (c.num_rows - 1) * a->ckv_row_stride * 2 + 1024},
              {a->k_pe, (c.num_rows - 1) * a->kpe_row_stride * 2 + 128},
              {a->prefix_len, 4ll * a->B},
              {a->anc, 8ll * a->B * a->Q},
              {a->group_start, a->G > 0 ? 4ll * (a->G + 1) : 0},
              {c.page_table, 4ll * a->B * c.max_pages}};
  for (const auto& in : ins)
    if (overlap(a->out, n * 512 * es, in.p, in.n) || overlap(a->lse, n * 4, in.p, in.n))
      return refuse(TV_ERR_INVALID_ARG, who, "an output overlaps an input");
  if (overlap(a->out, n * 512 * es, a->lse, n * 4) ||
      overlap(a->out, n * 512 * es, a->shared_len, 4ll * a->G) ||
      overlap(a->lse, n * 4, a->shared_len, 4ll * a->G))
    return refuse(TV_ERR_INVALID_ARG, who, "an output overlaps an input or the other output");
  return TV_OK;
}

}  // namespace

extern "C" {

int tv_rope_frequencies(const tv_rope_scaling* scaling, int rot_dim, double* frequencies,
                        double* magnitude) {
  tv::set_last_error("");
  const int rc = check_scaling(scaling, rot_dim, "tv_rope_frequencies");
  if (rc != TV_OK) return rc;
  if (!frequencies || !magnitude)
    return refuse(TV_ERR_INVALID_ARG, "tv_rope_frequencies", "NULL pointer");
  tv::rope_frequencies(*scaling, rot_dim, frequencies, magnitude);
  return TV_OK;
}

int tv_rope(const tv_rope_args* a, void* stream) {
  tv::set_last_error("");
  const int rc = check_rope(a);
  if (rc != TV_OK || a->T == 0) return rc;
  return result(tv::launch_rope_any(a, (cudaStream_t)stream), "tv_rope");
}

int tv_norm_rope(const tv_norm_rope_args* a, void* stream) {
  tv::set_last_error("");
  const int rc = check_norm_rope(a);
  if (rc != TV_OK || a->B == 0 || a->T == 0) return rc;
  return result(tv::launch_norm_rope(a, (cudaStream_t)stream), "tv_norm_rope");
}

size_t tv_shared_attn_workspace_size(const tv_shared_args* a) {
  tv::set_last_error("");
  return check_shared(a) == TV_OK && a->B > 0 ? tv::shared_workspace(a) : 0;
}

int tv_shared_attn(const tv_shared_args* a, void* workspace, size_t ws_bytes, void* stream) {
  tv::set_last_error("");
  const int rc = check_shared(a);
  if (rc != TV_OK || a->B == 0) return rc;
  if (!workspace || !aligned(workspace, 256) || ws_bytes < tv::shared_workspace(a))
    return refuse(TV_ERR_WORKSPACE, "tv_shared_attn",
                  "workspace missing, misaligned or smaller than tv_shared_attn_workspace_size()");
  return result(tv::launch_shared_attn(a, workspace, (cudaStream_t)stream), "tv_shared_attn");
}

int tv_token_sample(const tv_token_args* a, void* stream) {
  const char* who = "tv_token_sample";
  tv::set_last_error("");
  if (!a) return refuse(TV_ERR_INVALID_ARG, who, "args is NULL");
  if (a->struct_size != sizeof(tv_token_args))
    return refuse(TV_ERR_INVALID_ARG, who, "struct_size mismatch (ABI)");
  if (a->B < 0 || a->vocab < 1) return refuse(TV_ERR_INVALID_ARG, who, "bad B or vocab");
  if (a->vocab > (1 << 18)) return refuse(TV_ERR_UNSUPPORTED, who, "vocab > 2^18 not supported");
  if (a->B >= (1 << 24)) return refuse(TV_ERR_UNSUPPORTED, who, "B must be below 2^24");
  if (!type_ok(a->logits_dt)) return refuse(TV_ERR_INVALID_ARG, who, "logits must be F32 or BF16");
  if (a->logits_row_stride < a->vocab || a->logits_row_stride >= (1ll << 31))
    return refuse(TV_ERR_INVALID_ARG, who, "row stride below the row's size or past 2^31");
  if (a->B == 0) return TV_OK;
  if (!a->logits || !a->uniforms || !a->tokens)
    return refuse(TV_ERR_INVALID_ARG, who, "NULL pointer");
  const int64_t es = size_of(a->logits_dt), n = 4ll * a->B;
  if (!aligned(a->logits, es))
    return refuse(TV_ERR_INVALID_ARG, who, "logits not aligned to its element size");
  // the CTAs of a row read the inputs each for itself
  const struct {
    const void* p;
    int64_t n;
  } ins[6] = {{a->logits, ((a->B - 1) * a->logits_row_stride + a->vocab) * es},
              {a->temperature, n},
              {a->top_k, n},
              {a->top_p, n},
              {a->min_p, n},
              {a->uniforms, n}};
  for (const auto& in : ins)
    if (overlap(a->tokens, n, in.p, in.n) || overlap(a->kept, n, in.p, in.n))
      return refuse(TV_ERR_INVALID_ARG, who, "an output overlaps an input");
  if (overlap(a->tokens, n, a->kept, n))
    return refuse(TV_ERR_INVALID_ARG, who, "the outputs overlap");
  return result(tv::launch_token_sample(a, tv::current_sm_count(), (cudaStream_t)stream), who);
}

}  // extern "C"
