// kq_attn.cu -- host side of kq_attn_decode: the workspace's layout and the
// choice of the kernel (kq_attn_kernel.cuh).
#include "kq_attn_kernel.cuh"

namespace kq {

using namespace attn;

namespace {

// Query rows per pass over the cache: all T*G in one pass of 8, 16 or 32; more rows take several passes (heads of 256
// values: 16 at a time, whose sums already fill the registers).
int rows_per_pass(int head_dim, int rows) { return rows <= 8 ? 8 : rows <= 16 || head_dim > 128 ? 16 : 32; }

// Whether kq_attn_wide.cu takes the call, given bf16 queries and cache.
bool wide(int head_dim, int rows) { return rows > 16 && head_dim <= 128; }

struct Layout {
  int rows, RT;
  size_t count_off, ml_off, part_off, bytes;
};
Layout layout(int head_dim, int Hkv, int64_t T, int Hq, bool to_wide) {
  Layout L;
  const int R = static_cast<int>(T) * (Hq / Hkv);
  L.rows = to_wide ? kWideRows : rows_per_pass(head_dim, R);
  L.RT = R > 0 ? (R + L.rows - 1) / L.rows : 1;
  const size_t slots = 2 * static_cast<size_t>(num_sms()) * (to_wide ? 1 : 3);  // two parts per CTA, at most three CTAs per SM
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  // The counters, which have to be zero when a call begins, lie where no call writes anything else: one per range of the
  // most that any call cuts, whatever its sizes.  Parts are written before they are read.
  L.count_off = 0;
  L.ml_off = up(3 * static_cast<size_t>(num_sms()) * sizeof(int));
  L.part_off = L.ml_off + up(slots * L.rows * 2 * sizeof(float));
  L.bytes = L.part_off + up(slots * L.rows * head_dim * sizeof(float));
  return L;
}

}  // namespace

size_t attn_workspace_bytes(int head_dim, int Hkv, int64_t T, int Hq) {
  const size_t n = layout(head_dim, Hkv, T, Hq, false).bytes;
  if (!wide(head_dim, static_cast<int>(T) * (Hq / Hkv))) return n;
  const size_t m = layout(head_dim, Hkv, T, Hq, true).bytes;  // the size does not depend on the queries' type
  return n > m ? n : m;
}

cudaError_t launch_attn(const AttnArgs& a, int q_bf16, cudaStream_t st, AttnShape* ask) {
  const bool to_wide = q_bf16 && a.c.dtype == KQ_BF16 && wide(a.c.head_dim, a.T * a.G);
  const Layout L = layout(a.c.head_dim, a.c.n_kv_heads, a.T, a.Hq, to_wide);
  // the line of tiles is counted in 31 bits
  const int64_t tiles = ((a.max_pages << a.page_shift) + TK - 1) / TK + 8;  // 8: more than an item's start counts
  if (tiles * a.B > INT32_MAX / (a.c.n_kv_heads * L.RT)) return cudaErrorNotSupported;
  Params p;
  p.a = a;
  p.RT = L.RT;
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  p.count = reinterpret_cast<int*>(ws + L.count_off);
  p.part_ml = reinterpret_cast<float*>(ws + L.ml_off);
  p.part = reinterpret_cast<float*>(ws + L.part_off);
  if (to_wide) return launch_attn_wide(p, st, ask);
  if (a.c.dtype == KQ_BF16) return q_bf16 ? launch_attn_bf16_bf16(p, L.rows, st, ask) : launch_attn_bf16_f32(p, L.rows, st, ask);
  return q_bf16 ? launch_attn_f8_bf16(p, L.rows, st, ask) : launch_attn_f8_f32(p, L.rows, st, ask);
}

}  // namespace kq
