// Driver for the sanitizer build of the serving calls' C ABI (AddressSanitizer and
// UndefinedBehaviorSanitizer on the host code): every call with arguments that
// validation must refuse, or that ask for nothing, so that no kernel is launched.
// The pointers are fake, 16-byte aligned addresses that are never dereferenced.
// Exit 0: clean.
#include <stdint.h>
#include <stdio.h>

#include "kda.h"

namespace {

int failures = 0;

void expect(const char* what, kda_status got, kda_status want) {
  if (got != want) {
    fprintf(stderr, "serving sanitizer driver: %s returned %d, expected %d\n", what, (int)got, (int)want);
    ++failures;
  }
}

void* addr(int i, int off = 0) { return reinterpret_cast<void*>((uintptr_t(1) << 40) + (uintptr_t(i) << 36) + off); }
float* faddr(int i, int off = 0) { return static_cast<float*>(addr(i, off)); }
int* iaddr(int i, int off = 0) { return static_cast<int*>(addr(i, off)); }

}  // namespace

int main() {
  const kda_dtype BF = KDA_BF16, F = KDA_F32;
  auto norm = [&](int nm, long long qs, float eps, int n, int d, void* qo, long long qos) {
    return kda_qk_norm(addr(0), qs, addr(1), 4 * d, BF, (kda_norm)nm, faddr(2), nullptr, eps, 1.0f, iaddr(3), faddr(4), 16,
                       KDA_PAIR_HALVES, qo, qos, addr(6), 4 * d, BF, n, 8, 4, d, nullptr);
  };
  expect("norm kind", norm(9, 1024, 1e-6f, 10, 128, addr(5), 1024), KDA_ERR_DTYPE);
  expect("norm stride", norm(KDA_NORM_RMS, INT64_MAX, 1e-6f, 10, 128, addr(5), 1024), KDA_ERR_SHAPE);
  expect("norm negative stride", norm(KDA_NORM_RMS, INT64_MIN, 1e-6f, 10, 128, addr(5), 1024), KDA_ERR_SHAPE);
  expect("norm eps", norm(KDA_NORM_L2, 1024, -1.0f, 10, 128, addr(5), 1024), KDA_ERR_SHAPE);
  expect("norm size", norm(KDA_NORM_L2, 1024, 1e-6f, 10, 130, addr(5), 1024), KDA_ERR_UNSUPPORTED);
  expect("norm tokens", norm(KDA_NORM_L2, 1024, 1e-6f, INT32_MIN, 128, addr(5), 1024), KDA_ERR_SHAPE);
  expect("norm long stride", norm(KDA_NORM_L2, (1LL << 40) / 100000000 + 8, 1e-6f, 100000000, 16, addr(5), 128), KDA_ERR_SHAPE);
  expect("norm alias", norm(KDA_NORM_L2, 1024, 1e-6f, 10, 128, addr(0, 16), 1024), KDA_ERR_ALIAS);
  expect("norm nothing", norm(KDA_NORM_L2, 1024, 1e-6f, 0, 128, addr(5), 1024), KDA_OK);
  // tables
  expect("fork n", kda_cache_fork(iaddr(0), iaddr(1), iaddr(2), iaddr(3), iaddr(4), iaddr(5), INT32_MAX, 1, 8, 2, 16, nullptr),
         KDA_ERR_SHAPE);
  expect("fork table", kda_cache_fork(iaddr(0), iaddr(1), iaddr(2), iaddr(3), iaddr(4), iaddr(5), 4, 1, INT32_MAX, INT32_MAX, 16,
                                      nullptr), KDA_ERR_SHAPE);
  expect("fork alias", kda_cache_fork(iaddr(0), iaddr(1), iaddr(0), iaddr(3), iaddr(4), iaddr(5), 4, 1, 8, 2, 16, nullptr),
         KDA_ERR_ALIAS);
  expect("free n", kda_cache_free(iaddr(0), iaddr(1), iaddr(2), INT32_MAX, 8, 1 << 20, 16, nullptr), KDA_ERR_SHAPE);
  expect("free nothing", kda_cache_free(iaddr(0), iaddr(1), nullptr, 0, 8, 2, 16, nullptr), KDA_OK);
  expect("compact pages", kda_cache_compact(iaddr(0), iaddr(1), iaddr(0), iaddr(1), iaddr(4), iaddr(5), iaddr(6), 8, 2,
                                            INT32_MAX, nullptr), KDA_ERR_SHAPE);
  expect("compact null", kda_cache_compact(iaddr(0), iaddr(1), iaddr(0), iaddr(1), nullptr, iaddr(5), iaddr(6), 8, 2, 16,
                                           nullptr), KDA_ERR_NULL);
  expect("copy bytes", kda_cache_copy(addr(0), addr(0), SIZE_MAX, 1, 8, 8, iaddr(1), nullptr, 4, nullptr), KDA_ERR_SHAPE);
  expect("copy size", kda_cache_copy(addr(0), addr(0), (size_t)1 << 36, 65536, 65536, 65536, iaddr(1), nullptr, 4, nullptr),
         KDA_ERR_SHAPE);
  expect("copy alias", kda_cache_copy(addr(0), addr(0, 64), 64, 2, 8, 8, iaddr(1), nullptr, 4, nullptr), KDA_ERR_ALIAS);
  expect("copy nothing", kda_cache_copy(addr(0), addr(0), 64, 2, 8, 8, nullptr, nullptr, 0, nullptr), KDA_OK);
  // states on pages
  expect("paged B", kda_decode_step_paged(addr(0), addr(1), addr(2), BF, faddr(3), nullptr, nullptr, faddr(4), faddr(5), 9,
                                          iaddr(6), nullptr, addr(7), F, KDA_MAX_PAGED_SEQS + 1, 2, 128, 128, nullptr),
         KDA_ERR_SHAPE);
  expect("paged H", kda_decode_step_paged(addr(0), addr(1), addr(2), BF, faddr(3), nullptr, nullptr, faddr(4), faddr(5), 9,
                                          iaddr(6), nullptr, addr(7), F, 4, INT32_MAX, 128, 128, nullptr), KDA_ERR_SHAPE);
  expect("paged dtype", kda_decode_step_paged(addr(0), addr(1), addr(2), (kda_dtype)-4, faddr(3), nullptr, nullptr, faddr(4),
                                              faddr(5), 9, iaddr(6), nullptr, addr(7), F, 4, 2, 128, 128, nullptr),
         KDA_ERR_DTYPE);
  expect("verify K", kda_tree_verify(addr(0), addr(1), addr(2), BF, faddr(3), faddr(4), faddr(5), 9, iaddr(6), iaddr(7),
                                     nullptr, addr(8), F, faddr(9), 4, KDA_MAX_TREE + 1, 2, 128, 128, nullptr), KDA_ERR_SHAPE);
  expect("verify offsets", kda_tree_verify(addr(0), addr(1), addr(2), BF, faddr(3), faddr(4), faddr(5), 1, nullptr, iaddr(7),
                                           nullptr, addr(8), F, faddr(9), 1, 64, 1 << 20, 128, 128, nullptr), KDA_ERR_SHAPE);
  expect("verify alias", kda_tree_verify(addr(0), addr(1), addr(2), BF, faddr(3), faddr(4), faddr(5), 9, iaddr(6), iaddr(7),
                                         nullptr, addr(8), F, faddr(8, 64), 4, 8, 2, 128, 128, nullptr), KDA_ERR_ALIAS);
  expect("commit null", kda_tree_commit(addr(1), BF, faddr(3), faddr(9), iaddr(7), nullptr, nullptr, faddr(5), 9, iaddr(6),
                                        nullptr, 4, 8, 2, 128, 128, nullptr), KDA_ERR_NULL);
  expect("commit alias", kda_tree_commit(addr(1), BF, faddr(3), faddr(5), iaddr(7), nullptr, iaddr(8), faddr(5), 9, iaddr(6),
                                         nullptr, 4, 8, 2, 128, 128, nullptr), KDA_ERR_ALIAS);
  if (failures == 0) printf("clean\n");
  return failures != 0;
}
