// kq_attn.cu -- host side of kq_attn_decode: the workspace's layout and the
// choice of the kernel (kq_attn_kernel.cuh).
#include "kq_attn_kernel.cuh"

namespace kq {

using namespace attn;

namespace {

// Query rows per pass over the cache: all T*G in one pass of 8, 16 or 32; more rows take several passes (heads of 256
// values: 16 at a time, whose sums already fill the registers).
int rows_per_pass(int head_dim, int rows) { return rows <= 8 ? 8 : rows <= 16 || head_dim > 128 ? 16 : 32; }

struct Layout {
  int rows, RT;
  size_t count_off, ml_off, part_off, bytes;
};
Layout layout(int head_dim, int Hkv, int64_t B, int64_t T, int Hq) {
  Layout L;
  const int R = static_cast<int>(T) * (Hq / Hkv);
  L.rows = rows_per_pass(head_dim, R);
  L.RT = R > 0 ? (R + L.rows - 1) / L.rows : 1;
  const size_t slots = 2 * static_cast<size_t>(num_sms()) * 3;  // two parts per CTA, at most three CTAs per SM
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  L.count_off = 0;
  L.ml_off = up(static_cast<size_t>(B) * Hkv * L.RT * sizeof(int));
  L.part_off = L.ml_off + up(slots * L.rows * 2 * sizeof(float));
  L.bytes = L.part_off + up(slots * L.rows * head_dim * sizeof(float));
  return L;
}

}  // namespace

size_t attn_workspace_bytes(int head_dim, int Hkv, int64_t B, int64_t T, int Hq) {
  return layout(head_dim, Hkv, B, T, Hq).bytes;
}

cudaError_t launch_attn(const AttnArgs& a, int q_bf16, cudaStream_t st) {
  const Layout L = layout(a.c.head_dim, a.c.n_kv_heads, a.B, a.T, a.Hq);
  // the line of tiles is counted in 31 bits
  const int64_t tiles = ((a.max_pages << a.page_shift) + TK - 1) / TK + START + 1;
  if (tiles * a.B > INT32_MAX / (a.c.n_kv_heads * L.RT)) return cudaErrorNotSupported;
  Params p;
  p.a = a;
  p.RT = L.RT;
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  p.count = reinterpret_cast<int*>(ws + L.count_off);
  p.part_ml = reinterpret_cast<float*>(ws + L.ml_off);
  p.part = reinterpret_cast<float*>(ws + L.part_off);
  if (a.c.dtype == KQ_BF16) return q_bf16 ? launch_attn_bf16_bf16(p, L.rows, st) : launch_attn_bf16_f32(p, L.rows, st);
  return q_bf16 ? launch_attn_f8_bf16(p, L.rows, st) : launch_attn_f8_f32(p, L.rows, st);
}

}  // namespace kq
