// Driver for the sanitizer build of the attention layers' C ABI (AddressSanitizer and
// UndefinedBehaviorSanitizer on the host code): every call with arguments that validation
// must refuse, or that ask for nothing, so that no kernel is launched.  The pointers are
// fake, 16-byte aligned addresses that are never dereferenced.  Exit 0: clean.
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "kda.h"

namespace {

int failures = 0;

void expect(const char* what, kda_status got, kda_status want) {
  if (got != want) {
    fprintf(stderr, "attention sanitizer driver: %s returned %d, expected %d\n", what, (int)got, (int)want);
    ++failures;
  }
}

void* addr(int i, int off = 0) { return reinterpret_cast<void*>((uintptr_t(1) << 40) + (uintptr_t(i) << 36) + off); }
float* faddr(int i) { return static_cast<float*>(addr(i)); }
int* iaddr(int i, int off = 0) { return static_cast<int*>(addr(i, off)); }

}  // namespace

int main() {
  const kda_dtype BF = KDA_BF16, F = KDA_F32, E = KDA_E4M3;
  auto fwd = [&](int dt, long long qs, float scale, const int* cu, const int* cuk, int N, int nq, int nk, void* o, int hq, int hk, int dk) {
    return kda_attn_fwd(addr(0), qs, addr(1), 1024, addr(2), 1024, (kda_dtype)dt, scale, cu, cuk, N, nq, nk, o, 4096, BF, hq, hk, dk, 128, nullptr);
  };
  expect("fwd type", fwd(E, 4096, 1.0f, iaddr(3), nullptr, 2, 10, 10, addr(4), 32, 8, 128), KDA_ERR_DTYPE);
  expect("fwd any type", fwd(77, 4096, 1.0f, iaddr(3), nullptr, 2, 10, 10, addr(4), 32, 8, 128), KDA_ERR_DTYPE);
  expect("fwd counts", fwd(BF, 4096, 1.0f, iaddr(3), nullptr, INT32_MIN, INT32_MAX, INT32_MIN, addr(4), 32, 8, 128), KDA_ERR_SHAPE);
  expect("fwd heads", fwd(BF, 4096, 1.0f, iaddr(3), nullptr, 2, 10, 10, addr(4), INT32_MAX, INT32_MAX, 128), KDA_ERR_SHAPE);
  expect("fwd stride", fwd(BF, INT64_MAX, 1.0f, iaddr(3), nullptr, 2, 10, 10, addr(4), 32, 8, 128), KDA_ERR_SHAPE);
  expect("fwd negative stride", fwd(BF, INT64_MIN, 1.0f, iaddr(3), nullptr, 2, 10, 10, addr(4), 32, 8, 128), KDA_ERR_SHAPE);
  expect("fwd scale", fwd(BF, 4096, NAN, iaddr(3), nullptr, 2, 10, 10, addr(4), 32, 8, 128), KDA_ERR_SHAPE);
  expect("fwd size", fwd(BF, 4096, 1.0f, iaddr(3), nullptr, 2, 10, 10, addr(4), 32, 8, INT32_MAX), KDA_ERR_UNSUPPORTED);
  expect("fwd lists", fwd(BF, 4096, 1.0f, nullptr, iaddr(3), 2, 10, 10, addr(4), 32, 8, 128), KDA_ERR_NULL);
  expect("fwd alias", fwd(BF, 4096, 1.0f, iaddr(3), nullptr, 2, 10, 10, addr(1, 512), 32, 8, 128), KDA_ERR_ALIAS);
  expect("fwd nothing", fwd(BF, 4096, 1.0f, iaddr(3), iaddr(5), 2, 0, 10, addr(4), 32, 8, 128), KDA_OK);
  size_t n = 0;
  expect("page type", kda_kv_page_bytes(F, 64, 8, 128, 128, &n), KDA_ERR_DTYPE);
  expect("page tokens", kda_kv_page_bytes(E, INT32_MIN, 8, 128, 128, &n), KDA_ERR_UNSUPPORTED);
  expect("page heads", kda_kv_page_bytes(E, 64, INT32_MAX, 128, 128, &n), KDA_ERR_SHAPE);
  expect("page bytes", kda_kv_page_bytes(E, 128, KDA_MAX_HEADS, 128, 128, &n), KDA_OK);
  if (n != (size_t)KDA_MAX_HEADS * (128 * 256 + 8)) ++failures;
  auto append = [&](kda_dtype dt, kda_dtype kv, int pt, int pages, int rows, int width, int N, int total, int rot, int pairing, long long ks, void* pool) {
    return kda_kv_append(addr(0), ks, addr(1), 1024, addr(2), 4096, dt, nullptr, faddr(3), rot, (kda_pairing)pairing, addr(4), 4096, nullptr, 0,
                         pool, kv, pages, pt, iaddr(6), rows, width, iaddr(7), iaddr(8), iaddr(9), N, total, 32, 8, 128, 128, nullptr);
  };
  expect("append type", append(BF, F, 64, 9, 4, 4, 2, 10, 64, 0, 1024, addr(5)), KDA_ERR_DTYPE);
  expect("append pairing", append(BF, E, 64, 9, 4, 4, 2, 10, 64, -5, 1024, addr(5)), KDA_ERR_DTYPE);
  expect("append table", append(BF, E, 64, 9, INT32_MAX, INT32_MAX, 2, 10, 64, 0, 1024, addr(5)), KDA_ERR_SHAPE);
  expect("append tokens", append(BF, E, 64, 9, 4, 4, 2, INT32_MAX, 64, 0, 1024, addr(5)), KDA_ERR_SHAPE);
  expect("append page", append(BF, E, 1, 9, 4, 4, 2, 10, 64, 0, 1024, addr(5)), KDA_ERR_UNSUPPORTED);
  expect("append rotation", append(BF, E, 64, 9, 4, 4, 2, 10, INT32_MIN, 0, 1024, addr(5)), KDA_ERR_UNSUPPORTED);
  expect("append stride", append(BF, E, 64, 9, 4, 4, 2, 10, 64, 0, INT64_MIN, addr(5)), KDA_ERR_SHAPE);
  expect("append alias", append(BF, E, 64, KDA_MAX_PAGES, 4, 4, 2, 10, 64, 0, 1024, addr(0, -4096)), KDA_ERR_ALIAS);
  expect("append nothing", append(BF, E, 64, 9, 4, 4, 2, 0, 64, 0, 1024, addr(5)), KDA_OK);
  expect("read total", kda_kv_read(addr(0), E, 9, 64, iaddr(1), 4, 4, nullptr, nullptr, iaddr(2), addr(3), addr(4), BF, 2, INT32_MIN, 8, 128, 128, nullptr),
         KDA_ERR_SHAPE);
  expect("read alias", kda_kv_read(addr(0), E, 9, 64, iaddr(1), 4, 4, nullptr, nullptr, iaddr(2), addr(3), addr(3, 16), BF, 2, 10, 8, 128, 128, nullptr),
         KDA_ERR_ALIAS);
  expect("read nothing", kda_kv_read(addr(0), E, 9, 64, iaddr(1), 4, 4, nullptr, nullptr, nullptr, nullptr, nullptr, BF, 2, 0, 8, 128, 128, nullptr), KDA_OK);
  expect("plan width", kda_attn_decode_plan(E, 128, INT32_MAX, 4096, 16, 8, 8, 128, 128, &n), KDA_ERR_SHAPE);
  expect("plan", kda_attn_decode_plan(E, 128, 1 << 20, 4096, 16, 8, 8, 128, 128, &n), KDA_OK);
  auto decode = [&](float scale, int width, void* o, void* ws, size_t wn, int B, int K, int hq) {
    return kda_attn_decode(addr(0), BF, scale, addr(1), E, 9, 64, iaddr(2), 4, width, iaddr(3), iaddr(4), o, BF, ws, wn, B, K, hq, 8, 128, 128, nullptr);
  };
  expect("decode scale", decode(INFINITY, 4, addr(5), nullptr, 0, 2, 1, 32), KDA_ERR_SHAPE);
  expect("decode counts", decode(1.0f, 4, addr(5), nullptr, 0, INT32_MAX, INT32_MAX, 32), KDA_ERR_SHAPE);
  expect("decode workspace", decode(1.0f, 1 << 20, addr(5), nullptr, 0, 2, 1, 32), KDA_ERR_NULL);
  expect("decode small workspace", decode(1.0f, 1 << 20, addr(5), addr(6), 64, 2, 1, 32), KDA_ERR_SHAPE);
  expect("decode alias", decode(1.0f, 4, addr(0, 16), nullptr, 0, 2, 1, 32), KDA_ERR_ALIAS);
  expect("decode misaligned", decode(1.0f, 4, addr(5, 4), nullptr, 0, 2, 1, 32), KDA_ERR_MISALIGNED);
  if (failures) return 1;
  printf("clean\n");
  return 0;
}
