// tables_host.cpp - the index arithmetic of td_update_tables' kernel (td_internal.h) on a host
// without a GPU. For tests/test_tables_host.py.
#include "td_internal.h"

using namespace td;

extern "C" {

int64_t host_tables_grid(int n, int P, int max_slots, int sm_count) {
  TablesArgs a{};
  a.n = n;
  a.P = P;
  a.max_slots = max_slots;
  return tables_grid(a, sm_count);
}
// What a loop's index is after a step of the grid, and whether it then counts as below `end`.
int host_tables_goes_on(int64_t i, int64_t step, int64_t end) {
  TablesIndex at = static_cast<TablesIndex>(i);
  at += static_cast<TablesIndex>(step);
  return at < static_cast<TablesIndex>(end);
}
int host_pages_of(int len, int P) { return pages_of(len, P); }

}  // extern "C"
