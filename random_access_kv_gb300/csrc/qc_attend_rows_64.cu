// qc_attend_rows.cuh for heads of 64.
#define QC_ROWS_D 64
#include "qc_attend_rows.cuh"
