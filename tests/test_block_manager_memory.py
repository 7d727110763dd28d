"""The block manager's eviction step when the host runs out of memory: the call
answers PKV_ERR_NO_BLOCKS and leaves everything as it was (CPU only; a program
in which the n-th allocation fails, for every n)."""
import os
import subprocess

from paged_kv_cache_varlen_gb300 import build

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <new>
#include <vector>
#include "pkv.h"

static long fail_at = -1, count = 0;  // -1: no allocation fails
void* operator new(size_t n) {
  if (fail_at >= 0 && count++ == fail_at) throw std::bad_alloc();
  if (void* p = std::malloc(n)) return p;
  throw std::bad_alloc();
}
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, size_t) noexcept { std::free(p); }

struct State {
  std::vector<int32_t> words;
  explicit State(pkv_block_manager* bm, int blocks) {
    words.push_back(pkv_bm_num_free(bm));
    for (int b = 0; b < blocks; ++b) words.push_back(pkv_bm_refcount(bm, b));
    for (int64_t s = 1; s <= 3; ++s) {
      words.push_back((int32_t)pkv_bm_seq_len(bm, s));
      std::vector<int32_t> table(blocks);
      int32_t n = 0;
      if (pkv_bm_block_table(bm, s, table.data(), blocks, &n) != PKV_OK) std::abort();
      words.insert(words.end(), table.begin(), table.begin() + n);
    }
  }
};

int main() {
  const int blocks = 4096, bs = 4;
  int tried = 0;
  for (long n = 0;; ++n) {
    pkv_block_manager* bm = nullptr;
    if (pkv_bm_create(blocks, bs, nullptr, &bm) != PKV_OK) return 1;
    std::vector<int32_t> slots(8000);
    int32_t copies = 0;
    for (int64_t s = 1; s <= 2; ++s)
      if (pkv_bm_add_seq(bm, s) != PKV_OK ||
          pkv_bm_append(bm, s, 5000, slots.data(), nullptr, nullptr, 0, &copies) != PKV_OK)
        return 2;
    if (pkv_bm_fork(bm, 1, 3) != PKV_OK) return 3;  // shares all its blocks
    const State before(bm, blocks);
    const int64_t ids[3] = {2, 1, 3};
    const int32_t keep[3] = {40, 2000, 10};
    std::vector<int32_t> src(3 * 2000), dst(3 * 600);
    count = 0;
    fail_at = n;
    const pkv_status st = pkv_bm_evict_step(bm, ids, keep, 3, 2000, src.data(), 600, dst.data());
    const bool failed = count > n;
    fail_at = -1;
    if (failed) {
      ++tried;
      if (st != PKV_ERR_NO_BLOCKS || State(bm, blocks).words != before.words) {
        std::printf("allocation %ld: status %d, changed %d\n", n, st,
                    (int)(State(bm, blocks).words != before.words));
        return 4;
      }
      // and the same call, with memory, is right
      if (pkv_bm_evict_step(bm, ids, keep, 3, 2000, src.data(), 600, dst.data()) != PKV_OK)
        return 5;
    } else if (st != PKV_OK) {
      return 6;
    }
    // 10 + 500 + 3 blocks are taken, every other one is free, each once
    if (pkv_bm_num_free(bm) != blocks - 513) return 7;
    std::vector<int32_t> all(4 * (blocks - 513));
    if (pkv_bm_add_seq(bm, 9) != PKV_OK ||
        pkv_bm_append(bm, 9, (int32_t)all.size(), all.data(), nullptr, nullptr, 0, &copies) !=
            PKV_OK)
      return 8;
    for (int b = 0; b < blocks; ++b)
      if (pkv_bm_refcount(bm, b) != 1) return 9;
    pkv_bm_destroy(bm);
    if (!failed) break;
  }
  std::printf("%d failures\n", tried);
  return tried > 10 ? 0 : 10;
}
"""


def test_an_eviction_step_without_memory_changes_nothing(tmp_path):
    source, program = tmp_path / "p.cpp", tmp_path / "p"
    source.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", os.path.join(build.ROOT, "include"),
                    str(source), os.path.join(build.CSRC, "block_manager.cpp"), "-o",
                    str(program)], check=True, capture_output=True)
    r = subprocess.run([str(program)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, (r.returncode, r.stdout)
