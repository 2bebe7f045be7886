// wd_call: the entry points of a decode step with their arguments in one block.
// ctypes takes 80 ns per argument: 1.9 us for wd_block_norm's 22, 0.6 us as a block. On
// the host a small call takes 5.9 instead of 7.6 us (norm), 4.4 instead of 5.3 (matvec),
// 6.6 instead of 7.8 (attend).
#include <cstdint>
#include <cstring>

#include "wd_block.cuh"

namespace {

// The next argument.
struct Args {
  const char* at;
  explicit Args(const void* args) : at(static_cast<const char*>(args)) {}
  int64_t word() {
    int64_t v;
    std::memcpy(&v, at, 8);
    at += 8;
    return v;
  }
  bool wide = false;  // an argument of 32 bits does not fit them
  int32_t i32() {
    const int64_t v = word();
    wide |= v != (int32_t)v;
    return (int32_t)v;
  }
  float f32() {
    double v;
    std::memcpy(&v, at, 8);
    at += 8;
    return (float)v;
  }
  template <typename T>
  T* ptr() {
    return reinterpret_cast<T*>((uintptr_t)word());
  }
};

}  // namespace

extern "C" moe_status wd_call(int32_t which, const void* args) {
  if (!args) return wd::refuse(MOE_ERR_NULL, "wd_call: arguments are required");
  Args a(args);
  auto refused = [] { return wd::refuse(MOE_ERR_SHAPE, "wd_call: an argument does not fit its 32 bits"); };
  // (each read on its own: the order in which a call's operands are evaluated is open)
  switch (which) {
    case WD_CALL_FP4_MATVEC: {
      auto* s = a.ptr<const wd_fp4_shape>();
      auto *pc = a.ptr<const uint8_t>(), *ps = a.ptr<const uint8_t>();
      auto* x = a.ptr<const void>();
      const int32_t xt = a.i32();
      const int64_t ldx = a.word();
      const int32_t B = a.i32();
      auto* y = a.ptr<void>();
      const int32_t yt = a.i32();
      const int64_t ldy = a.word();
      if (a.wide) return refused();
      return wd_fp4_matvec(s, pc, ps, x, xt, ldx, B, y, yt, ldy, a.ptr<void>());
    }
    case WD_CALL_KV4_APPEND:
    case WD_CALL_KV4_GATHER: {
      auto* c = a.ptr<const wd_kv4_cache>();
      auto *k = a.ptr<void>(), *v = a.ptr<void>();
      const int32_t type = a.i32();
      const int64_t ldk = a.word(), ldv = a.word();
      const int32_t T = a.i32();
      auto* table = a.ptr<const int32_t>();
      const int32_t blocks = a.i32();
      auto *lens = a.ptr<const int32_t>(), *cu = a.ptr<const int32_t>();
      const int32_t S = a.i32();
      auto* err = a.ptr<int32_t>();
      auto* st = a.ptr<void>();
      if (a.wide) return refused();
      return which == WD_CALL_KV4_APPEND ? wd_kv4_append(c, k, v, type, ldk, ldv, T, table, blocks, lens, cu, S, err, st)
                                         : wd_kv4_gather(c, k, v, type, ldk, ldv, T, table, blocks, lens, cu, S, err, st);
    }
    case WD_CALL_KV4_ATTEND: {
      auto* c = a.ptr<const wd_kv4_cache>();
      auto* q = a.ptr<const void>();
      const int32_t type = a.i32();
      const int64_t ldq = a.word();
      const int32_t S = a.i32(), heads = a.i32();
      auto* table = a.ptr<const int32_t>();
      const int32_t blocks = a.i32();
      auto* lens = a.ptr<const int32_t>();
      const float scale = a.f32();
      const int32_t window = a.i32();
      auto* out = a.ptr<void>();
      const int64_t ldo = a.word();
      auto* lse = a.ptr<float>();
      auto* work = a.ptr<void>();
      const size_t bytes = (size_t)a.word();
      auto* err = a.ptr<int32_t>();
      if (a.wide) return refused();
      return wd_kv4_attend(c, q, type, ldq, S, heads, table, blocks, lens, scale, window, out, ldo, lse, work, bytes,
                           err, a.ptr<void>());
    }
    case WD_CALL_BLOCK_NORM: {
      const int32_t T = a.i32(), H = a.i32();
      auto* res = a.ptr<const void>();
      const int32_t rt = a.i32();
      const int64_t ldr = a.word();
      auto* y = a.ptr<const void>();
      const int32_t yt = a.i32();
      const int64_t ldy = a.word();
      auto *post = a.ptr<const void>(), *pre = a.ptr<const void>(), *gate = a.ptr<const void>();
      const int32_t wt = a.i32();
      const int64_t gate_ld = a.word();
      const int32_t gate_step = a.i32();
      const float res_scale = a.f32(), eps = a.f32();
      auto* res_out = a.ptr<void>();
      const int64_t ldro = a.word();
      auto* out = a.ptr<void>();
      const int32_t ot = a.i32();
      const int64_t ldo = a.word();
      if (a.wide) return refused();
      return wd_block_norm(T, H, res, rt, ldr, y, yt, ldy, post, pre, gate, wt, gate_ld, gate_step, res_scale, eps,
                           res_out, ldro, out, ot, ldo, a.ptr<void>());
    }
    case WD_CALL_ROPE: {
      auto* r = a.ptr<const wd_rotation>();
      auto* x = a.ptr<const void>();
      const int32_t type = a.i32();
      const int64_t ldx = a.word();
      const int32_t T = a.i32(), heads = a.i32(), dim = a.i32();
      auto* positions = a.ptr<const int32_t>();
      auto* out = a.ptr<void>();
      const int64_t ldo = a.word();
      if (a.wide) return refused();
      return wd_rope(r, x, type, ldx, T, heads, dim, positions, out, ldo, a.ptr<void>());
    }
    case WD_CALL_KV4_ROPE_APPEND: {
      auto* c = a.ptr<const wd_kv4_cache>();
      auto* r = a.ptr<const wd_rotation>();
      auto* q = a.ptr<const void>();
      const int64_t ldq = a.word();
      const int32_t heads = a.i32();
      auto* q_out = a.ptr<void>();
      const int64_t ldqo = a.word();
      auto *k = a.ptr<const void>(), *v = a.ptr<const void>();
      const int32_t type = a.i32();
      const int64_t ldk = a.word(), ldv = a.word();
      const int32_t T = a.i32();
      auto* table = a.ptr<const int32_t>();
      const int32_t blocks = a.i32();
      auto *lens = a.ptr<const int32_t>(), *cu = a.ptr<const int32_t>();
      const int32_t S = a.i32();
      auto* err = a.ptr<int32_t>();
      if (a.wide) return refused();
      return wd_kv4_rope_append(c, r, q, ldq, heads, q_out, ldqo, k, v, type, ldk, ldv, T, table, blocks, lens, cu, S, err,
                                a.ptr<void>());
    }
    case WD_CALL_KV4_ATTEND_CHUNK: {
      auto* c = a.ptr<const wd_kv4_cache>();
      auto* q = a.ptr<const void>();
      const int32_t type = a.i32();
      const int64_t ldq = a.word();
      const int32_t T = a.i32(), heads = a.i32();
      auto* table = a.ptr<const int32_t>();
      const int32_t blocks = a.i32();
      auto *lens = a.ptr<const int32_t>(), *cu = a.ptr<const int32_t>();
      const int32_t S = a.i32();
      const float scale = a.f32();
      const int32_t window = a.i32();
      auto* out = a.ptr<void>();
      const int64_t ldo = a.word();
      auto* lse = a.ptr<float>();
      auto* work = a.ptr<void>();
      const size_t bytes = (size_t)a.word();
      auto* err = a.ptr<int32_t>();
      if (a.wide) return refused();
      return wd_kv4_attend_chunk(c, q, type, ldq, T, heads, table, blocks, lens, cu, S, scale, window, out, ldo, lse, work,
                                 bytes, err, a.ptr<void>());
    }
  }
  return wd::refuse(MOE_ERR_UNSUPPORTED, "wd_call: no such entry point");
}
