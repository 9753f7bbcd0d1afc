// kq_attn.cu -- host side of kq_attn_decode: the workspace's layout and the
// choice of the kernel (kq_attn_kernel.cuh).
#include "kq_attn_kernel.cuh"

namespace kq {

using namespace attn;

namespace {

// Query rows per pass over the cache: all T*G in one pass of 8, 16 or 32; more rows take several passes (heads of 256
// values: 16 at a time, whose sums already fill the registers).
int rows_per_pass(int head_dim, int rows) { return rows <= 8 ? 8 : rows <= 16 || head_dim > 128 ? 16 : 32; }

// Whether kq_attn_wide.cu can take a call with bf16 queries and cache.
bool could_be_wide(int head_dim, int rows) { return rows > 16 && head_dim <= 128; }

// Whether it does, heads being the sequences times their key-value heads.  Its one CTA per SM reads a head's cache once for
// 128 rows; the other kernel goes over it for every 32 rows (17 to 32 rows: once, too).  But a head split over many CTAs is
// joined by one of them, and a part of 128 rows is four times as much to join.  So beyond 32 rows it takes the call from
// three heads' tiles per 16 rows on, or half as many where the table has room for long caches (the lengths themselves are
// not known here).  Measured in us, this kernel's time / the other's, up to 1500 and up to 6007 positions:
//   heads of 128:  4 heads    8         16        32        64
//     32 rows     31/35 47/80  31/37 33/57  24/38 31/47  20/31 35/49  23/30 49/56   (256 heads 55/56)
//     64 rows     51/37 84/57  52/38 54/44  37/31 45/47  26/28 42/58  28/38 54/82
//    128 rows     94/38 158/44 95/30 97/45  65/28 75/55  41/37 61/86  43/54 74/139
// and up to 24000 positions, 128 rows: 16 heads 111/148, 8 heads 116/94, 4 heads 154/70.
// Heads of 64 are half the bytes: 17 to 32 rows pay up to 32 heads (32 rows up to 6007 positions: 25/37 at 8 heads,
// 28/32 at 32, 41/40 at 64, 70/60 at 128).
bool wide(int head_dim, int rows, int64_t heads, int64_t room) {
  if (!could_be_wide(head_dim, rows)) return false;
  if (rows <= 32) return head_dim == 128 || heads <= 32;
  const int64_t tiles = heads * ((rows + kWideRows - 1) / kWideRows);
  return (room > 16384 ? 32 : 16) * tiles >= 3 * (rows < kWideRows ? rows : kWideRows);
}

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
  if (!could_be_wide(head_dim, static_cast<int>(T) * (Hq / Hkv))) return n;
  const size_t m = layout(head_dim, Hkv, T, Hq, true).bytes;  // the size depends on neither B nor the queries' type
  return n > m ? n : m;
}

cudaError_t launch_attn(const AttnArgs& a, int q_bf16, cudaStream_t st, AttnShape* ask) {
  const bool to_wide = q_bf16 && a.c.dtype == KQ_BF16 && wide(a.c.head_dim, a.T * a.G, static_cast<int64_t>(a.B) * a.c.n_kv_heads, a.room);
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
